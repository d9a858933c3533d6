"""Serving-pass operators on the GPU where lengths, scores and values reach
the ends of their types, and in kernel variants that need many keys."""
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import bit_weight_quantized_awq_amd as awq  # noqa: E402

DEV = "cuda:0"
MOST = 2 ** 31 - 1


def say(msg):
    print(f"\n[case] {msg}", flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    awq.lib()
    yield


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).to(DEV)


def num(t):
    return t.detach().cpu().numpy()


# ------------------------------------------------------------------------------- batch_layout
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("B,large", [(4, [0, 1]), (5, [0, 1, 2, 3, 4]), (300, list(range(20, 300))),
                                     (700, [300, 301, 302]), (1500, [3, 700, 1400, 1401])])
def test_layout_sums_past_32_bits(B, large, tree):
    """Token counts whose sums pass 2^31: held there, and every token that
    there is room for is placed as in 64 bits."""
    say(f"batch_layout sums past 32 bits B={B} tree={tree}")
    T, W, bs, F = 600, 2, 16, 40
    cached = np.full(B, 9, dtype=np.int64)
    counts = 1 + np.arange(B, dtype=np.int64) % 3
    counts[large] = MOST - np.arange(len(large))
    held = np.ones(B, dtype=np.int64)
    start = np.concatenate([[0], np.cumsum(counts)])
    table = np.full((B, W), -1, dtype=np.int32)
    table[:, 0] = 100 + np.arange(B)
    parents = np.array([-1 if t % 5 == 0 else 0 for t in range(T)], dtype=np.int32)
    dev = i32(table)
    got = awq.batch_layout(i32(cached), i32(counts), i32(held), i32(np.arange(F)), dev, bs, 2000, T,
                           parents=i32(parents) if tree else None, mask_words=1)
    np.testing.assert_array_equal(num(got.q_start), np.minimum(start, MOST))
    need = -(-(cached + counts) // bs) - held
    fit = np.minimum(need, W - 1)
    gained = np.minimum(np.maximum(F - (np.cumsum(fit) - fit), 0), fit)
    np.testing.assert_array_equal(num(got.blocks_held), held + gained)
    np.testing.assert_array_equal(num(got.status), np.minimum(
        [gained.sum(), (need - gained).sum(), start[-1], (cached + counts).max()], MOST))
    table[:, 1] = np.where(gained > 0, np.cumsum(gained) - 1, -1)
    np.testing.assert_array_equal(num(dev), table)
    t = np.arange(T)
    b = np.searchsorted(start, t, side="right") - 1
    inside = t < start[-1]
    b = np.where(inside, b, 0)
    i = t - start[b]
    first = parents if tree else i - 1
    # Here a parent is none or the request's token 0, itself a root.
    depth = np.where((first >= 0) & (first < i), 1, 0) if tree else i
    at = cached[b] + i
    page = np.where(at // bs < W, table[b, np.minimum(at // bs, W - 1)], -1)
    np.testing.assert_array_equal(num(got.requests), np.where(inside, b, -1))
    np.testing.assert_array_equal(num(got.positions), np.where(inside, cached[b] + depth, 0))
    np.testing.assert_array_equal(num(got.slots),
                                  np.where(inside & (page >= 0), page * bs + at % bs, -1))
    for x in np.flatnonzero(inside):
        want = {int(i[x])} if tree else set(range(int(i[x]) + 1))
        if tree and depth[x]:
            want.add(0)
        bits = int(num(got.tree_mask)[x, 0]) & (2 ** 64 - 1)
        assert bits == sum(1 << w for w in want if w < 64), x


def test_layout_positions_past_32_bits():
    say("batch_layout positions past 32 bits")
    got = awq.batch_layout(i32([MOST - 1, MOST]), i32([4, 2]), i32([MOST, 0]), i32([0]),
                           i32([[5], [6]]), 16, 8, 6)
    np.testing.assert_array_equal(num(got.positions), [MOST - 1] + [MOST] * 5)
    np.testing.assert_array_equal(num(got.slots), [-1] * 6)
    assert num(got.status)[3] == MOST


# ------------------------------------------------------------------------------- host threads
def test_host_threads_on_one_stream():
    """Attention split over work-groups and products split along K from four
    host threads on one stream, through one workspace: the same bits as from
    one thread."""
    import threading

    import awq_inputs
    say("host threads on one stream")
    gen = torch.Generator(DEV).manual_seed(0)

    def rand(*shape):
        return torch.randn(shape, generator=gen, device=DEV).to(torch.float16)

    def attention(ctx, n, heads, kvh):
        blocks = -(-(ctx + n) // 16)
        kc, vc, q = rand(blocks, 16, kvh, 128), rand(blocks, 16, kvh, 128), rand(n, heads, 128)
        table, cached, start = i32([list(range(blocks))]), i32([ctx]), i32([0, n])
        return lambda: awq.tree_attention(q, kc, vc, table, cached, start)

    def product(M, K, N):
        p = awq_inputs.make_inputs(M, K, N, 128, seed=M)
        x, w, z, s = (torch.from_numpy(p[k]).to(DEV) for k in ("x", "qweight", "qzeros", "scales"))
        return lambda: awq.gemm(x, w, z, s, None, 128)

    calls = [attention(3000, 3, 8, 2), attention(5000, 40, 32, 8), product(16, 14336, 4096),
             product(1, 8192, 7168)]
    want = [f() for f in calls]
    torch.cuda.synchronize()
    wrong, failed = [], []

    def work(x):
        try:
            for _ in range(30):
                if not torch.equal(calls[x](), want[x]):
                    wrong.append(x)
        except Exception as e:   # reported by the thread that waits
            failed.append(e)

    threads = [threading.Thread(target=work, args=(x,)) for x in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    torch.cuda.synchronize()
    assert not failed and not wrong and not any(t.is_alive() for t in threads), (failed, wrong)


# ----------------------------------------------------------------------------- tree_attention
from test_gpu_serving import E4M3, HALF, TINY, Problem, wide  # noqa: E402

F16, BF16 = torch.float16, torch.bfloat16
# (heads, key heads, contexts, tokens): 16, 32 and 128 rows of a key head, runs
# of many tiles that several work-groups join.
ROWS = [(4, 2, [700, 3, 90], [2, 1, 3]), (8, 2, [2500, 40], [6, 4]), (32, 2, [1500, 0], [9, 5])]


def fill(p, k, v):
    """Keys and values (rows in the order of the requests, heads, D) into the cache."""
    slots = [p.table[b, j // p.bs] * p.bs + j % p.bs for b in range(len(p.ctx))
             for j in range(p.ctx[b] + p.added[b])]
    one = None if p.k_scale is None else torch.ones(p.kvh, device=DEV)
    awq.kv_write(k.to(p.dtype), v.to(p.dtype), i32(slots), p.kc, p.vc, one, one)
    if one is not None:
        p.k_scale, p.v_scale = one, one


@pytest.mark.parametrize("heads,kvh,ctx,added", ROWS)
@pytest.mark.parametrize("dtype,e4m3", [(F16, False), (BF16, False), (F16, True), (BF16, True)])
@pytest.mark.parametrize("scale", [2.0 ** 16, -2.0 ** 22, 2.0 ** 26, 2.0 ** 100])
def test_attention_huge_scores(heads, kvh, ctx, added, dtype, e4m3, scale):
    """Scores that are exact and so far apart that the largest ones alone have
    weights: the mean of their values, however large the scores are.

    Whole numbers below 16 in the queries and keys: every product and sum is
    exact in float32, and scores that differ do so by 2^16 at least, where
    float32's step at the largest (2^16 times 16 * 16 * 64) is 2^7 of the
    same.  Equal scores have equal weights.  What is left is the rounding of
    the sum of up to `ties` values, of the quotient and of the output."""
    p = Problem(ctx, added, heads, kvh, 64, 16, dtype, e4m3, tree=True, seed=heads)
    say(f"huge scores heads={heads}/{kvh} {dtype} e4m3={e4m3} scale={scale}")
    rng = np.random.default_rng(heads)
    rows = sum(ctx) + sum(added)
    k, v = (torch.from_numpy(rng.integers(-15, 16, (rows, kvh, 64))).to(torch.float32).to(DEV)
            for _ in range(2))
    fill(p, k, v)
    p.q[:] = torch.from_numpy(rng.integers(-15, 16, p.q.shape)).to(dtype).to(DEV)
    got = wide(p.run(scale=scale))
    kc, vc, q = wide(p.kc), wide(p.vc), wide(p.q)
    bs, G = p.bs, heads // kvh
    for b in range(len(ctx)):
        j = np.arange(ctx[b] + added[b])
        page, off = p.table[b, j // bs], j % bs
        for t in range(p.q_start[b], p.q_start[b + 1]):
            bits = int(p.mask[t, 0])
            see = (j < ctx[b]) | np.array([bool(bits >> int(max(x - ctx[b], 0)) & 1) for x in j])
            for h in range(heads):
                s = (kc[page, off, h // G] @ q[t, h]) * np.sign(scale)
                best = see & (s == s[see].max())
                x = vc[page, off, h // G][best]
                want, size = x.mean(0), np.abs(x).mean(0)
                lim = len(x) * 2.0 ** -22 * size + HALF[dtype] * 1.01 * np.abs(want) + TINY[dtype]
                assert (np.abs(got[t, h] - want) <= lim).all(), (b, t, h, got[t, h][:4], want[:4])


@pytest.mark.parametrize("heads,kvh,ctx,added", ROWS)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_attention_scores_of_minus_infinity(heads, kvh, ctx, added, dtype):
    """Keys that overflowed to a score of -infinity: a row that sees nothing
    else is NaN, as the softmax of its scores; beside finite scores they have
    no weight; a row that sees nothing at all stays 0."""
    p = Problem(ctx, added, heads, kvh, 64, 16, dtype, tree=True, seed=heads + 1)
    say(f"scores of -infinity heads={heads}/{kvh} {dtype}")
    p.q[:, :, 0] = 1.0
    last = len(ctx) - 1
    for b in range(len(ctx)):
        for j in range(ctx[b] + added[b]):
            if b == 0 and j % 7 == 0:
                continue
            p.kc[int(p.table[b, j // 16]), j % 16, :, 0] = float("-inf")
    if ctx[last] == 0:
        p.mask[p.q_start[last]] = 0
    got = wide(p.run())
    out, weight, spread, keys = p.want()
    assert (keys > 0)[:p.q_start[last]].all()
    other = np.arange(p.T) >= p.q_start[1]
    nothing = keys == 0
    assert (got[nothing] == 0).all()
    assert np.isnan(out[other & ~nothing]).all()
    assert np.isnan(got[other & ~nothing]).all()
    first = slice(0, p.q_start[1])
    assert np.isfinite(got[first]).all()
    # As Problem.bound, with the spread of the finite scores.
    spread = np.full_like(spread, 64 * 12.0 * 6.0 * p.scale)
    lim = p.bound(out, weight, spread, keys)
    assert (np.abs(got - out)[first] <= lim[first]).all()


@pytest.mark.parametrize("heads,kvh,ctx,added", ROWS)
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("drafted", [False, True])
def test_attention_infinite_value_without_weight(heads, kvh, ctx, added, dtype, drafted):
    """An infinite value whose key scores -infinity: 0 * infinity is NaN in its
    channel for the rows that see it, and nothing for the others."""
    p = Problem(ctx, added, heads, kvh, 64, 16, dtype, tree=True, seed=heads + 2)
    say(f"infinite value without weight heads={heads}/{kvh} {dtype} drafted={drafted}")
    p.q[:, :, 0] = 1.0
    i = added[0] // 2
    j = ctx[0] + i if drafted else 37
    page, off = int(p.table[0, j // 16]), j % 16
    p.kc[page, off, :, 0] = float("-inf")
    p.vc[page, off, :, 5] = float("inf")
    got = wide(p.run())
    sees = np.zeros(p.T, dtype=bool)
    for t in range(added[0]):
        sees[t] = not drafted or bool((int(p.mask[t, 0]) >> i) & 1)
    assert sees.any() and not sees.all()
    assert np.isnan(got[sees][:, :, 5]).all()
    assert np.isfinite(np.delete(got, 5, axis=2)).all()
    assert np.isfinite(got[~sees]).all()


@pytest.mark.parametrize("heads,kvh,ctx,added", ROWS)
@pytest.mark.parametrize("scale,size", [(0.0, 1e18), (1e-38, 4e18), (-3e-38, 4e18), (1e-41, 1e18),
                                        (1e-60, 1e18)])
def test_attention_smallest_scales(heads, kvh, ctx, added, scale, size):
    """Scales at and near zero over bfloat16 products of up to 1e38.

    Errors: as Problem.bound; a scale below 2^-126 is a multiple of 2^-149, so
    scores move by half of that times the product, at most 2^-150 * 64 *
    size^2, and a zero scale counts as 2^-149."""
    p = Problem(ctx, added, heads, kvh, 64, 16, BF16, tree=True, seed=heads + 3)
    say(f"scale {scale} products of {size * size}")
    p.kc.mul_(size)
    p.q.copy_(torch.nan_to_num(p.q * (size / 8)))
    p.scale = scale
    got = wide(p.run(scale=scale))
    out, weight, spread, keys = p.want()
    small = 0.0
    if abs(scale) < 2.0 ** -126:
        top = np.nanmax(np.abs(wide(p.kc))) * np.abs(wide(p.q)).max() * 64
        small = 2.0 ** -148 * 1.45 * top
        assert small < 1e-4
    assert np.isfinite(got).all()
    lim = p.bound(out, weight, spread, keys) + 2 * small * weight
    assert (np.abs(got - out) <= lim).all(), np.abs(got - out).max()
    if scale != 0 and abs(scale) > 1e-40:
        assert np.abs(out - wide(p.run(scale=0.0))).max() > 0.1   # the scale matters


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("bs,tree", [(16, True), (24, True), (64, False)])
def test_attention_32_rows_over_long_contexts(D, dtype, e4m3, bs, tree):
    """17 to 32 rows of a key head on average: waves go over many tiles, and
    row blocks are split over work-groups and joined."""
    added = [5, 6, 7, 5]
    assert 16 < sum(added) * 4 / len(added) <= 32
    Problem([4100, 37, 1900, 6], added, 8, 2, D, bs, dtype, e4m3, tree=tree, seed=D + bs).check(
        f"32 rows D={D} {dtype} e4m3={e4m3} bs={bs} tree={tree}")


class Sampled:
    """A long problem whose rows are checked for some of its heads only.
    Errors are bounded as in Problem.bound."""

    def __init__(self, ctx, added, heads, D, bs, dtype, e4m3, seed):
        gen = torch.Generator(DEV).manual_seed(seed)
        self.dtype, self.ctx, self.added, self.D, self.bs = dtype, ctx, added, D, bs
        used = [-(-(c + n) // bs) for c, n in zip(ctx, added)]
        blocks = sum(used) + 3
        ids = np.random.default_rng(seed).permutation(blocks)
        self.table = np.full((len(ctx), max(used)), -1, dtype=np.int32)
        at = 0
        for b, u in enumerate(used):
            self.table[b, :u] = ids[at:at + u]
            at += u

        def rand(*shape):
            return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float16)

        self.kc, self.vc = (rand(blocks, bs, heads, D).to(E4M3 if e4m3 else dtype) for _ in range(2))
        self.q = rand(sum(added), heads, D).to(dtype)
        self.q_start = np.concatenate([[0], np.cumsum(added)]).astype(np.int32)
        self.heads = heads

    def check(self, what, sample):
        from oracle import serving_oracle as ref
        say(what)
        got = wide(awq.tree_attention(self.q, self.kc, self.vc, i32(self.table), i32(self.ctx),
                                      i32(self.q_start)))[:, sample]
        assert np.isfinite(got).all()
        part = Problem.__new__(Problem)
        part.D, part.dtype, part.v_scale = self.D, self.dtype, None
        part.vc = self.vc[:, :, sample]
        out, weight, spread, keys = ref.tree_attention(
            wide(self.q[:, sample]), wide(self.kc[:, :, sample]), wide(part.vc), self.table, self.ctx,
            self.q_start, None, self.D ** -0.5)
        lim = part.bound(out, weight, spread, keys)
        bad = np.abs(got - out) > lim
        assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist())


@pytest.mark.parametrize("D,dtype,e4m3,bs", [
    (64, F16, False, 16), (64, BF16, False, 16), (128, F16, True, 16), (64, F16, True, 32),
    (64, F16, False, 24), (128, BF16, True, 20), (256, F16, False, 8)])
def test_attention_runs_of_many_steps(D, dtype, e4m3, bs):
    """As many key heads as work-groups and more than 32 rows of each, so one
    work-group goes over a whole context: more steps than pages are looked up
    for at once (64 steps of 64 or 128 keys), with pages that hold whole
    groups of keys and pages that do not."""
    heads = 256
    step = 128 if D == 64 and e4m3 else 64
    ctx = [64 * step * 2 + 300, 50]
    Sampled(ctx, [35, 34], heads, D, bs, dtype, e4m3, seed=D + bs).check(
        f"many steps D={D} {dtype} e4m3={e4m3} bs={bs}", [0, 7, 255])


def test_layout_trees_of_many_requests():
    """More requests than threads keep in registers (four of 256 threads), with
    trees, masks of two words and a capacity that cuts the last ones."""
    from oracle import serving_oracle as ref
    from test_gpu_serving import random_parents
    say("batch_layout trees of 1500 requests")
    B = 1500
    rng = np.random.default_rng(1)
    cached, added = rng.integers(0, 200, B), rng.integers(0, 9, B)
    added[[3, 700, 1499]] = [90, 1, 130]
    held = -(-cached // 16)
    table = np.full((B, 24), -1, dtype=np.int32)
    ids = rng.permutation(40000).astype(np.int32)
    at = 0
    for b in range(B):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
    free = ids[at:at + 1200]
    T = int(added.sum()) - 7
    parents = random_parents(rng, added)[:T]
    want = ref.batch_layout(cached, added, held, free, 5, table, 16, 40000, T, parents, 2)
    t = i32(table)
    got = awq.batch_layout(i32(cached), i32(added), i32(held), i32(free), t, 16, 40000, T,
                           parents=i32(parents), mask_words=2, free_start=i32([5]))
    np.testing.assert_array_equal(num(t), want["block_table"])
    for key in ("q_start", "slots", "positions", "requests", "blocks_held", "status", "tree_mask"):
        np.testing.assert_array_equal(num(getattr(got, key)), want[key], err_msg=key)
