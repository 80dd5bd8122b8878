"""Attention over a paged cache on the GPU against 64 bits.

Tolerances.  With e = 2^-24: a score of d products in fp32 is off by (d + 8) 2 e of the sum of their sizes at most (the
tensor core cuts its partial sums off instead of rounding them, hence the 2), which is the relative error x of its weight;
the maximum and the sum cancel out of it but for x of the largest.  The sum of n weights adds (n + 64) e.  bf16 weights
are rounded, 2^-8 of each.  An output is off by the weights' errors on sum_j p_j |v_j|, and by its own rounding u."""
import random

import pytest
import torch

pytestmark = pytest.mark.gpu

E = 2.0 ** -24


@pytest.fixture(scope="module")
def tp():
    from tensor_transformer_mlp_tma_gb300 import tpmlp
    return tpmlp


def tree_of(n, rng, words):
    """Random drafts: each token's own bit and those of the tokens above it, as `words` signed words."""
    of = []
    for i in range(n):
        above = rng.randint(-1, i - 1)
        of.append((of[above] if above >= 0 else 0) | 1 << i)
    return [[(m >> 64 * w & (1 << 64) - 1) - (1 << 64 if m >> 64 * w + 63 & 1 else 0) for w in range(words)] for m in of]


class Problem:
    """`lens`: (cached, new) tokens of each sequence."""

    def __init__(self, lens, heads, kv, d, page, dt, tree=False, order="heads", seed=0, tail=0, spread=1.0, spare=3):
        g = torch.Generator(device="cpu").manual_seed(seed)
        rng = random.Random(seed)
        self.lens, self.heads, self.kv, self.d, self.page, self.dt = lens, heads, kv, d, page, dt
        counts = [(c + n + page - 1) // page for c, n in lens]
        pages = sum(counts) + spare
        shape = (pages, page, kv, d) if order == "tokens" else (pages, kv, page, d)
        K, V = (torch.randn(shape, generator=g) for _ in "kv")
        self.T = sum(n for _, n in lens) + tail
        Q = spread * torch.randn(self.T, heads, d, generator=g)
        self.K, self.V = (x.to(dt).cuda().transpose(1, 2) if order == "tokens" else x.to(dt).cuda() for x in (K, V))
        self.Q = Q.to(dt).cuda()
        free = list(range(pages))
        rng.shuffle(free)
        # entries past a sequence's pages hold no page
        table = torch.full((len(lens), max(counts + [1]) + 1), -12345, dtype=torch.int32)
        for b, c in enumerate(counts):
            for i in range(c):
                table[b, i] = free.pop()
        self.free = free
        self.table = table.cuda()
        self.q_start = torch.tensor([sum(n for _, n in lens[:b]) for b in range(len(lens) + 1)], dtype=torch.int32).cuda()
        self.kv_len = torch.tensor([c + n for c, n in lens], dtype=torch.int32).cuda()
        self.tree = None
        if tree:
            words = max(1, (max([n for _, n in lens] + [1]) + 63) // 64)
            rows = [r for _, n in lens for r in tree_of(n, rng, words)] + [[-1] * words] * tail
            self.tree = torch.tensor(rows, dtype=torch.int64).reshape(self.T, words).cuda()

    def run(self, tp, algo=None, ctx=None, O=None, **kw):
        cache = tp.KvCache.of(self.K, self.V)
        self.ctx = ctx or tp.CacheAttnContext(self.T, len(self.lens), self.heads, self.kv, self.d, self.dt,
                                              algo=tp.ALGO_DEFAULT if algo is None else algo, **kw)
        return tp.cache_attention(self.ctx, cache, self.Q, self.q_start, self.kv_len, self.table, self.tree, O)

    def seen(self, b, device="cuda"):
        """[new, keys]: what each new token of sequence b sees."""
        c, n = self.lens[b]
        m = torch.ones(n, c + n, dtype=torch.bool, device=device)
        if self.tree is None:
            m[:, c:] = torch.ones(n, n, dtype=torch.bool, device=device).tril()
        else:
            q0 = sum(x for _, x in self.lens[:b])
            j = torch.arange(n, device=device)
            words = self.tree[q0:q0 + n].to(device)
            inside = j < 64 * words.shape[1]
            j = j.clamp(max=64 * words.shape[1] - 1)
            m[:, c:] = (words[:, j // 64] >> (j % 64) & 1).bool() & inside
        return m

    def check(self, O, scale=None):
        scale = self.d ** -0.5 if scale is None else scale
        q0 = 0
        for b, (c, n) in enumerate(self.lens):
            keys = torch.arange(c + n, device="cuda")
            page = self.table[b].long()[keys // self.page]
            K, V = (x[page, :, keys % self.page].double() for x in (self.K, self.V))  # [keys, kv, d]
            seen = self.seen(b)
            G = self.heads // self.kv
            for h in range(self.kv):
                Q = self.Q[q0:q0 + n, h * G:(h + 1) * G].double().reshape(n * G, self.d)
                mask = seen.repeat_interleave(G, 0)
                k, v = K[:, h], V[:, h]
                used = mask.any(0)
                k, v = torch.where(used[:, None], k, 0.0), torch.where(used[:, None], v, 0.0)
                S = (Q @ k.t() * scale).masked_fill(~mask, -float("inf"))
                P = torch.softmax(S, 1).nan_to_num(0.0)
                ref = P @ v
                size = P @ v.abs()
                x = 2 * (self.d + 8) * 2 * E * ((Q.abs() @ k.abs().t()) * abs(scale) * mask).amax(1, keepdim=True) if c + n else 0.0
                u = torch.finfo(self.dt).eps / 2
                tol = u * ref.abs() + (x + (c + n + 64) * E + (2.0 ** -8 if self.dt == torch.bfloat16 else 0.0)) * 1.01 * size
                got = O[q0:q0 + n, h * G:(h + 1) * G].double().reshape(n * G, self.d)
                bad = ~((got - ref).abs() <= tol)
                assert not bool(bad.any()), (b, h, int(bad.sum()), float((got - ref).abs().max()))
            q0 += n


CASES = [  # lens, heads, kv, d, page, tree
    ([(0, 1)], 1, 1, 64, 16, False), ([(1, 1)], 2, 1, 128, 16, False), ([(0, 5)], 4, 4, 64, 8, False),
    ([(127, 1)], 8, 8, 128, 16, False), ([(128, 1)], 8, 2, 128, 16, False), ([(129, 3)], 8, 2, 128, 16, True),
    ([(2047, 1)], 32, 32, 128, 16, False), ([(5000, 1)], 16, 2, 128, 64, False), ([(1000, 64)], 8, 1, 128, 16, True),
    ([(300, 1), (0, 0), (5, 1), (1111, 1), (64, 1), (63, 1), (0, 1), (777, 1)], 8, 2, 64, 16, False),
    ([(0, 0), (10, 17), (3, 0), (600, 33), (129, 9), (0, 0)], 16, 4, 128, 32, True),
    ([(0, 300)], 4, 2, 128, 64, False), ([(100, 257), (0, 130), (31, 1)], 12, 4, 64, 16, False),
    ([(40, 70)], 6, 2, 80, 8, True), ([(513, 100)], 8, 8, 256, 16, True), ([(513, 4), (90, 2)], 16, 2, 256, 48, False),
    ([(200, 20)], 5, 5, 96, 24, True), ([(77, 5)], 6, 3, 192, 16, False), ([(1000, 1)], 64, 1, 128, 128, False),
    ([(100, 1)] * 70, 4, 1, 32, 16, False), ([(3, 2)] * 300, 2, 2, 8, 8, False), ([(250, 7)], 40, 8, 128, 256, True),
    ([(20000, 2)], 8, 1, 64, 16, False), ([(90, 65)], 3, 1, 72, 40, True), ([(50, 129)], 2, 2, 128, 16, True),
    ([(383, 1), (384, 1), (385, 1)], 17, 1, 128, 16, False), ([(700, 16)], 8, 1, 128, 16, False),
]


@pytest.mark.parametrize("i", range(len(CASES)))
@pytest.mark.parametrize("kind", ["bf16", "bf16-ffma", "f32"])
def test_against_64_bits(tp, kind, i):
    lens, heads, kv, d, page, tree = CASES[i]
    p = Problem(lens, heads, kv, d, page, torch.float32 if kind == "f32" else torch.bfloat16, tree, seed=i,
                order="tokens" if i % 3 == 2 else "heads", tail=i % 2 * 3)
    O = torch.full((p.T, heads, d), 5.0, dtype=p.dt, device="cuda")
    p.run(tp, tp.ALGO_SIMT if kind == "bf16-ffma" else None, O=O)
    assert tp.check_device_status(p.ctx) == tp.OK
    p.check(O)
    # rows behind the last sequence stay
    assert bool((O[p.T - i % 2 * 3:] == 5).all())
    # the same bits again, from a workspace that is left ready
    assert torch.equal(p.run(tp, ctx=p.ctx), O) if not i % 2 else True


@pytest.mark.parametrize("page,d", [(1, 64), (3, 128), (20, 64), (7, 40)])
def test_pages_of_any_size(tp, page, d):
    for dt in (torch.bfloat16, torch.float32):
        p = Problem([(100, 3), (17, 2)], 4, 2, d, page, dt, True, seed=page)
        p.check(p.run(tp))
        assert tp.check_device_status(p.ctx) == tp.OK


@pytest.mark.parametrize("seed", range(24))
def test_random_shapes(tp, seed):
    rng = random.Random(seed)
    kv = rng.choice((1, 2, 3, 8))
    heads = kv * rng.choice((1, 2, 3, 4, 8, 16))
    d = rng.choice((8, 32, 64, 80, 96, 128, 128, 136, 192, 256))
    most = rng.choice((1, 1, 8, 70, 200))
    lens = [(rng.choice((0, 1, 15, 16, 127, 128, 500, rng.randint(0, 3000))), rng.randint(0, most)) for _ in range(rng.randint(1, 20))]
    dt = torch.float32 if seed % 4 == 3 else torch.bfloat16
    p = Problem(lens, heads, kv, d, rng.choice((8, 16, 16, 32, 48, 64, 128)), dt, rng.random() < 0.5, seed=seed, tail=rng.randint(0, 3))
    O = torch.full((p.T, heads, d), 5.0, dtype=dt, device="cuda")
    p.check(p.run(tp, O=O))
    assert tp.check_device_status(p.ctx) == tp.OK


@pytest.mark.parametrize("kind", ["bf16", "bf16-ffma", "f32"])
@pytest.mark.parametrize("lens,heads,kv,d", [([(200, 20)], 8, 2, 128), ([(100, 3), (5, 7)], 4, 4, 64), ([(130, 90)], 8, 4, 256),
                                             ([(120, 40)], 4, 2, 128), ([(0, 100)], 2, 2, 64)])
def test_what_is_not_seen_has_no_part(tp, kind, lens, heads, kv, d):
    """NaN and infinities in rows behind a sequence's end, in drafts of other branches and in pages of nobody."""
    p = Problem(lens, heads, kv, d, 16, torch.float32 if kind == "f32" else torch.bfloat16, True, seed=3)
    algo = tp.ALGO_SIMT if kind == "bf16-ffma" else None
    clean = p.run(tp, algo)
    p.check(clean)
    for page in p.free:
        p.K[page] = float("nan")
        p.V[page] = float("inf")
    q0 = 0
    bad_of = []
    for b, (c, n) in enumerate(lens):
        end = (c + n + 15) // 16 * 16
        for key in range(c + n, end):
            p.K[int(p.table[b, key // 16]), :, key % 16] = float("nan")
            p.V[int(p.table[b, key // 16]), :, key % 16] = float("nan") if key % 2 else float("-inf")
        # one draft that some tokens see and others do not
        seen = p.seen(b)[:, c:]
        j = next(i for i in range(n) if 0 < int(seen[:, i].sum()) < n)
        p.V[int(p.table[b, (c + j) // 16]), 0, (c + j) % 16, :5] = float("inf")
        p.K[int(p.table[b, (c + j) // 16]), kv - 1, (c + j) % 16, 1] = float("nan")
        bad_of.append((q0, seen[:, j]))
        q0 += n
    O = p.run(tp, algo)
    assert tp.check_device_status(p.ctx) == tp.OK
    G = heads // kv
    for (q0, sees), (c, n) in zip(bad_of, lens):
        rows, ref = O[q0:q0 + n], clean[q0:q0 + n]
        tol = 2.0 ** -6 if p.dt == torch.bfloat16 else 1e-5
        # who sees it has what it does: infinity in five components, NaN in the heads of the key
        hit = rows[sees]
        if kv > 1:
            assert bool((hit[:, :G, :5] == float("inf")).all())
            assert torch.allclose(hit[:, :G, 5:].float(), ref[sees][:, :G, 5:].float(), atol=tol, rtol=tol)
        assert bool(hit[:, (kv - 1) * G:].isnan().all())
        # who does not, has the value of before
        assert torch.allclose(rows[~sees].float(), ref[~sees].float(), atol=tol, rtol=tol)


def test_rows_that_see_nothing(tp):
    for dt in (torch.bfloat16, torch.float32):
        p = Problem([(0, 20), (150, 9)], 4, 2, 64, 16, dt, True, seed=4)
        p.tree[3] = 0
        p.tree[25] = 0  # sees the cached keys alone
        O = p.run(tp)
        assert bool((O[3] == 0).all())
        p.check(O)


def test_long_drafts_past_the_tree(tp):
    """Drafts past the bits of the tree are seen by nobody."""
    p = Problem([(30, 70)], 4, 2, 64, 16, torch.bfloat16, True, seed=5)
    p.tree = p.tree[:, :1].contiguous()
    p.check(p.run(tp))


@pytest.mark.parametrize("spread,scale", [(30.0, None), (1e4, None), (1.0, 4.0), (0.0, None), (1.0, -0.5), (1.0, 0.0)])
def test_scores_far_apart(tp, spread, scale):
    """Weights of one key alone, and the running maximum growing by much; even weights; scores turned round."""
    for dt in (torch.bfloat16, torch.float32):
        p = Problem([(700, 5), (1500, 1)], 8, 2, 128, 16, dt, True, seed=6, spread=spread)
        # scores that grow along the sequence: the reference changes again and again
        p.check(p.run(tp, scale=scale), scale)


def test_growing_scores(tp):
    """Every tile's largest score is above all before it."""
    for dt in (torch.bfloat16, torch.float32):
        p = Problem([(3000, 2)], 4, 1, 64, 16, dt, True, seed=7)
        p.Q[:, :, 0] = 8.0
        pos = torch.arange(3002, device="cuda")
        page = p.table[0].long()[pos // 16]
        p.K[page, 0, pos % 16, 0] = (0.125 * pos).to(dt)
        p.check(p.run(tp))
        p.K[page, 0, pos % 16, 0] = (-0.125 * pos).to(dt)
        p.check(p.run(tp))


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_bad_lengths_and_pages_are_reported(tp, kind):
    dt = torch.float32 if kind == "f32" else torch.bfloat16
    lens = [(50, 2), (40, 3), (20, 1), (60, 2)]

    def problem():
        return Problem(lens, 4, 2, 64, 16, dt, seed=8)

    p = problem()
    p.kv_len[1] = 2  # fewer keys than new tokens
    O = p.run(tp)
    assert tp.check_device_status(p.ctx) == tp.ERR_INVALID_ARG and bool((O[2:5] == 0).all())
    good = problem()
    ref = good.run(tp)
    assert torch.equal(O[:2], ref[:2]) and torch.equal(O[5:], ref[5:])
    for value in (-1, 1 << 20):
        p = problem()
        p.kv_len[2] = value
        O = p.run(tp)
        assert tp.check_device_status(p.ctx) == tp.ERR_INVALID_ARG and bool((O[5] == 0).all())
    for start in (-4, 1 << 20):
        p = problem()
        p.q_start[2] = start
        O = p.run(tp)
        assert tp.check_device_status(p.ctx) == tp.ERR_INVALID_ARG and torch.equal(O[:2], ref[:2])
    for page in (-1, p.K.shape[0], -(1 << 31), (1 << 31) - 1):
        p = problem()
        p.table[3, 1] = page  # keys 16 .. 31 of the last sequence
        O = p.run(tp)
        assert int(p.ctx.workspace[4:8].view(torch.int32)[0]) == 3
        assert tp.check_device_status(p.ctx) == tp.ERR_INVALID_ARG and torch.equal(O[:6], ref[:6])
        q = problem()
        at = int(q.table[3, 1])
        q.K[at], q.V[at] = 0.0, 0.0
        q.check(O)


def test_no_sequences_and_no_tokens(tp):
    for batch, T in ((0, 0), (3, 0), (0, 4)):
        ctx = tp.CacheAttnContext(T, batch, 4, 2, 64, torch.bfloat16)
        cache = tp.KvCache(2, 16, 2, 64, torch.bfloat16)
        i32 = dict(dtype=torch.int32, device="cuda")
        O = torch.full((T, 4, 64), 5.0, dtype=torch.bfloat16, device="cuda")
        tp.cache_attention(ctx, cache, O.clone(), torch.zeros(batch + 1, **i32), torch.zeros(batch, **i32),
                           torch.zeros(batch, 1, **i32), O=O)
        assert bool((O == 5).all()) and tp.check_device_status(ctx) == tp.OK


def test_other_streams_and_replays_with_other_lengths(tp):
    for dt in (torch.bfloat16, torch.float32):
        p = Problem([(900, 1), (30, 1), (0, 1), (2000, 1)], 16, 4, 128, 16, dt, seed=9)
        want = p.run(tp)
        torch.cuda.synchronize()
        st = torch.cuda.Stream()
        with torch.cuda.stream(st):
            got = p.run(tp, ctx=p.ctx)
        st.synchronize()
        assert torch.equal(got, want)
        cache = tp.KvCache.of(p.K, p.V)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            O = tp.cache_attention(p.ctx, cache, p.Q, p.q_start, p.kv_len, p.table)
        for lens in ([(900, 1), (30, 1), (0, 1), (2000, 1)], [(3, 1), (31, 1), (0, 1), (1024, 1)], [(500, 1), (0, 1), (0, 1), (0, 1)]):
            p.kv_len.copy_(torch.tensor([c + n for c, n in lens], dtype=torch.int32))
            graph.replay()
            torch.cuda.synchronize()
            p.lens = lens
            p.check(O)
        assert tp.check_device_status(p.ctx) == tp.OK


def test_pages_shared_and_given_twice(tp):
    """Sequences with a common beginning share its pages."""
    p = Problem([(100, 1), (100, 4), (64, 2)], 8, 2, 128, 16, torch.bfloat16, seed=10)
    p.table[1, :4] = p.table[0, :4]
    p.table[2, :4] = p.table[0, 0]
    p.check(p.run(tp))


def test_a_cache_past_32_bits(tp):
    for dt in (torch.bfloat16, torch.float32):
        p = Problem([(70, 2), (33, 1)], 4, 2, 128, 64, dt, True, seed=11)
        pages = 140000 if dt == torch.bfloat16 else 70000  # past 2^31 elements or bytes
        K, V = (torch.empty(pages, 2, 64, 128, dtype=dt, device="cuda") for _ in "kv")
        far = [pages - 1, pages - 3, 5]
        for b, (c, n) in enumerate(p.lens):
            for i in range((c + n + 63) // 64):
                old, new = int(p.table[b, i]), far.pop()
                K[new], V[new] = p.K[old], p.V[old]
                p.table[b, i] = new
        p.K, p.V = K, V
        p.check(p.run(tp))


def test_a_long_sequence(tp):
    p = Problem([(131072, 4)], 8, 1, 128, 64, torch.bfloat16, True, seed=12)
    p.check(p.run(tp))


def test_a_step_of_serving(tp):
    """Tokens of a prompt, then drafts, appended and attended to, give what one pass over all of them gives."""
    heads, kv, d, dt = 8, 2, 64, torch.bfloat16
    n, chunk = 200, [130, 1, 69]
    g = torch.Generator(device="cpu").manual_seed(13)
    QKV = torch.randn(n, (heads + 2 * kv) * d, generator=g).to(dt).cuda()
    gains = [(1 + 0.1 * torch.randn(d, generator=g)).to(dt).cuda() for _ in "qk"]
    rope = tp.RopeTable(d)
    pos = torch.arange(n, device="cuda")
    cache = tp.KvCache(16, 16, kv, d, dt)
    order = torch.randperm(16, generator=g)
    table = order.int().cuda()[None]
    slot = order.cuda()[pos // 16] * 16 + pos % 16
    out = []
    done = 0
    for m in chunk:
        r = slice(done, done + m)
        ctx = tp.QkContext(m, heads, kv, d, dt, rope)
        Q = tp.kv_append(ctx, cache, QKV[r], pos[r], slot[r], *gains)
        done += m
        i32 = dict(dtype=torch.int32, device="cuda")
        actx = tp.CacheAttnContext(m, 1, heads, kv, d, dt)
        out.append(tp.cache_attention(actx, cache, Q, torch.tensor([0, m], **i32), torch.tensor([done], **i32), table))
        assert tp.check_device_status(ctx) == tp.OK and tp.check_device_status(actx) == tp.OK
    ctx = tp.QkContext(n, heads, kv, d, dt, rope)
    Q, K = tp.qk_forward(ctx, QKV, pos, *gains)
    V = QKV[:, -kv * d:].view(n, kv, d)
    p = Problem([(0, n)], heads, kv, d, 16, dt)
    p.Q, p.table = Q, table
    p.K, p.V = cache.K, cache.V
    assert torch.equal(cache.K[order.cuda()[pos // 16], :, pos % 16], K) and torch.equal(cache.V[order.cuda()[pos // 16], :, pos % 16], V)
    p.check(torch.cat(out))
