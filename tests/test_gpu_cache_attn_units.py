"""Attention over a paged cache where it is divided: units of few rows and of many, one or several per sequence, cut between
blocks, in one tile of keys or in many; against 64 bits, with the tolerances of test_gpu_cache_attn."""
import pytest
import torch

import test_gpu_cache_attn as base
from test_gpu_cache_attn import Problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tp():
    from tensor_transformer_mlp_tma_gb300 import tpmlp
    return tpmlp


# few rows per sequence on average, but long ones among them; many on average, but short ones among them
FEW = [([(100, 1)] * 60 + [(500, 150)], 8, 2), ([(0, 200)] + [(300, 1)] * 40, 4, 4), ([(3, 0)] * 90 + [(1000, 70), (0, 5)], 16, 2),
       ([(127, 1), (128, 1), (129, 1)], 8, 1), ([(5000, 32)], 3, 3), ([(4000, 8), (0, 1)], 12, 4)]
MANY = [([(1000, 200), (3, 1), (0, 0), (127, 1)], 8, 2), ([(0, 65)], 2, 2), ([(63, 65)], 2, 2), ([(64, 65)], 2, 2),
        ([(200, 128)], 5, 5), ([(200, 129)], 5, 5), ([(20000, 33)], 4, 1), ([(250, 9), (300, 40)], 16, 2), ([(10, 3)] * 12, 33, 1),
        ([(3000, 300), (1000, 17)], 6, 2)]


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("d", [24, 64, 128, 136, 256])
@pytest.mark.parametrize("i", range(len(FEW) + len(MANY)))
def test_units(tp, i, d, tree):
    lens, heads, kv = (FEW + MANY)[i]
    p = Problem(lens, heads, kv, d, (16, 8, 64)[i % 3], torch.bfloat16, tree, seed=100 + i, order="tokens" if i % 2 else "heads", tail=2)
    O = torch.full((p.T, heads, d), 5.0, dtype=p.dt, device="cuda")
    p.run(tp, O=O)
    assert tp.check_device_status(p.ctx) == tp.OK
    p.check(O)
    assert bool((O[p.T - 2:] == 5).all())
    assert torch.equal(p.run(tp, ctx=p.ctx, O=O.clone()), O)


@pytest.mark.parametrize("lens,heads,kv,d", [([(200, 6), (5, 7)], 8, 2, 256), ([(130, 30)] + [(20, 2)] * 20, 4, 2, 128),
                                             ([(1000, 50)], 8, 2, 64), ([(300, 70), (100, 90)], 4, 2, 256), ([(0, 130)], 2, 2, 136)])
def test_what_is_not_seen_has_no_part(tp, lens, heads, kv, d):
    base.test_what_is_not_seen_has_no_part(tp, "bf16", lens, heads, kv, d)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_rows_that_see_nothing(tp, d):
    p = Problem([(0, 150), (150, 30), (0, 70)], 4, 2, d, 16, torch.bfloat16, True, seed=4)
    p.tree[:40] = 0      # a whole unit's and more
    p.tree[149] = 0
    p.tree[155] = 0      # sees the cached keys alone
    p.tree[185:187] = 0
    O = p.run(tp)
    assert bool((O[:40] == 0).all()) and bool((O[149] == 0).all()) and bool((O[185:187] == 0).all())
    p.check(O)


@pytest.mark.parametrize("spread,scale", [(30.0, None), (1e4, None), (1.0, 4.0), (0.0, None), (1.0, -0.5), (1.0, 0.0)])
@pytest.mark.parametrize("d", [128, 256])
def test_scores_far_apart(tp, spread, scale, d):
    p = Problem([(700, 50), (1500, 20)], 8, 2, d, 16, torch.bfloat16, True, seed=6, spread=spread)
    p.check(p.run(tp, scale=scale), scale)


@pytest.mark.parametrize("d", [64, 136])
def test_growing_scores(tp, d):
    p = Problem([(3000, 40)], 4, 1, d, 16, torch.bfloat16, True, seed=7)
    p.Q[:, :, 0] = 8.0
    pos = torch.arange(3040, device="cuda")
    page = p.table[0].long()[pos // 16]
    for sign in (1, -1):
        p.K[page, 0, pos % 16, 0] = (sign * 0.125 * pos).to(p.dt)
        p.check(p.run(tp))


def test_bad_lengths_are_reported(tp):
    lens = [(500, 100), (400, 150), (0, 80)]
    ref = Problem(lens, 4, 2, 128, 16, torch.bfloat16, seed=8).run(tp)
    for value in (149, -1, 1 << 20):
        p = Problem(lens, 4, 2, 128, 16, torch.bfloat16, seed=8)
        p.kv_len[1] = value
        O = p.run(tp)
        assert tp.check_device_status(p.ctx) == tp.ERR_INVALID_ARG and bool((O[100:250] == 0).all())
        assert torch.equal(O[:100], ref[:100]) and torch.equal(O[250:], ref[250:])
    # the same context serves the next call
    p.kv_len[1] = 550
    assert torch.equal(p.run(tp, ctx=p.ctx), ref) and tp.check_device_status(p.ctx) == tp.OK
    # a page that is none counts as zeros
    p.table[2, 1] = -1
    O = p.run(tp, ctx=p.ctx)
    assert tp.check_device_status(p.ctx) == tp.ERR_INVALID_ARG and torch.equal(O[:250], ref[:250])
    q = Problem(lens, 4, 2, 128, 16, torch.bfloat16, seed=8)
    at = int(q.table[2, 1])
    q.K[at], q.V[at] = 0.0, 0.0
    q.check(O)


def test_replays_with_other_lengths(tp):
    """A graph captured for one division of the work is replayed for others: one token per sequence, and prompts."""
    lens = [[(900, 1), (30, 1), (0, 1), (2000, 217)], [(3, 217), (31, 1), (0, 1), (1024, 1)], [(500, 55)] * 4, [(0, 0), (2000, 0), (5, 220), (0, 0)]]
    for heads in (4, 2):  # 55 and 28 rows per sequence
        p = Problem(lens[0], heads, 2, 128, 16, torch.bfloat16, seed=9)
        p.table = torch.arange(4 * 141, dtype=torch.int32, device="cuda").reshape(4, 141)
        g = torch.Generator(device="cpu").manual_seed(9)
        p.K, p.V = (torch.randn(4 * 141, 2, 16, 128, generator=g).to(p.dt).cuda() for _ in "kv")
        p.run(tp)
        cache = tp.KvCache.of(p.K, p.V)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            O = tp.cache_attention(p.ctx, cache, p.Q, p.q_start, p.kv_len, p.table)
        for now in lens + lens[:1]:
            p.lens = now
            p.kv_len.copy_(torch.tensor([c + n for c, n in now], dtype=torch.int32))
            p.q_start.copy_(torch.tensor([sum(n for _, n in now[:b]) for b in range(5)], dtype=torch.int32))
            graph.replay()
            torch.cuda.synchronize()
            p.check(O)
        assert tp.check_device_status(p.ctx) == tp.OK


def test_two_calls_at_once(tp):
    """Two contexts on two streams, whose calls run beside one another."""
    a = Problem([(3000, 100), (20, 40)], 8, 2, 128, 16, torch.bfloat16, seed=10)
    b = Problem([(2000, 1)] * 9, 8, 2, 128, 16, torch.bfloat16, seed=11)
    want = [a.run(tp), b.run(tp)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in "ab"]
    got = [[], []]
    for _ in range(8):
        for i, p in enumerate((a, b)):
            with torch.cuda.stream(streams[i]):
                got[i].append(p.run(tp, ctx=p.ctx))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x, want[i]) for x in got[i])


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_caches_of_any_alignment(tp, dt):
    """Rows that do not begin on 16 bytes, and strides that are odd: read element by element."""
    for cut in (1, 3):
        p = Problem([(200, 20), (33, 1)], 4, 2, 64, 16, dt, True, seed=12)
        wide = [torch.full((x.shape[0], 2, 16, 64 + cut), float("nan"), dtype=dt, device="cuda") for x in (p.K, p.V)]
        for w, x in zip(wide, (p.K, p.V)):
            w[..., cut:] = x
        p.K, p.V = (w[..., cut:] for w in wide)
        p.check(p.run(tp))
        assert tp.check_device_status(p.ctx) == tp.OK


def test_keys_and_values_in_one_array(tp):
    """K and V of a page next to one another: [pages, 2, kv, page, d]."""
    p = Problem([(700, 70), (100, 5)], 8, 2, 128, 16, torch.bfloat16, seed=13)
    both = torch.stack((p.K, p.V), 1).contiguous()
    p.K, p.V = both[:, 0], both[:, 1]
    p.check(p.run(tp))


def test_a_captured_step_of_serving(tp):
    """kv_append and cache_attention in one graph, replayed token after token, give what one call for all tokens does."""
    heads, kv, d, dt, first, steps = 8, 2, 128, torch.bfloat16, 120, 20
    g = torch.Generator(device="cpu").manual_seed(14)
    n = first + steps
    QKV = torch.randn(n, (heads + 2 * kv) * d, generator=g).to(dt).cuda()
    gains = [(1 + 0.1 * torch.randn(d, generator=g)).to(dt).cuda() for _ in "qk"]
    rope = tp.RopeTable(d)
    i32 = dict(dtype=torch.int32, device="cuda")

    def pass_of(T, cache, table):
        ctx = tp.QkContext(T, heads, kv, d, dt, rope)
        attn = tp.CacheAttnContext(T, 1, heads, kv, d, dt)
        x, pos = torch.empty(T, QKV.shape[1], dtype=dt, device="cuda"), torch.empty(T, dtype=torch.int64, device="cuda")
        slot, q_start, kv_len = torch.empty_like(pos), torch.tensor([0, T], **i32), torch.zeros(1, **i32)

        def feed(at):
            x.copy_(QKV[at:at + T])
            pos.copy_(torch.arange(at, at + T))
            slot.copy_(table[0].long()[pos // 16] * 16 + pos % 16)
            kv_len.fill_(at + T)

        def run():
            return tp.cache_attention(attn, cache, tp.kv_append(ctx, cache, x, pos, slot, *gains), q_start, kv_len, table)

        return feed, run, (ctx, attn)

    table = torch.randperm(12, generator=g).int().cuda()[None]
    cache = tp.KvCache(12, 16, kv, d, dt)
    feed, run, _ = pass_of(n, cache, table)
    feed(0)
    want = run().clone()

    cache = tp.KvCache(12, 16, kv, d, dt)
    feed, run, _ = pass_of(first, cache, table)
    feed(0)
    out = [run()]
    feed, run, contexts = pass_of(1, cache, table)
    feed(first)
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        O = run()
    for i in range(steps):
        feed(first + i)
        graph.replay()
        out.append(O.clone())
    torch.cuda.synchronize()
    assert all(tp.check_device_status(c) == tp.OK for c in contexts)
    # weights and outputs rounded (2^-8 each) in either pass, of values whose weighted sizes are below 6
    assert float((torch.cat(out).float() - want.float()).abs().max()) < 2 * 2 * 2.0 ** -8 * 6
