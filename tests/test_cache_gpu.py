"""GPU tests of the paged cache's append and attention against the fp64 oracle.

Tolerance of the attention, elementwise, u = eps/2 of the type (bf16 2^-8,
fp16 2^-11), a = sum_j p_j |v_j|: the weights are rounded to the type before the
product with v (u a), the output once (u |o|); the weights' own error in fp32:
exponentials within 7.5e-5, scores of D fp32-accumulated products within
scale D 2^-23 sum|q k| <= 1.3e-4 for these inputs (sum|q k| <= 130 at D = 128),
each entering numerator and sum: 4e-4 a in all.  The log-sum-exp: 2.1e-4.
Tolerance of the append: that of the rotation (1e-6 of the pair's magnitude
before, here with the norm's factor and its own 1e-6) and one rounding."""
import numpy as np
import pytest
import torch

import joint_text_image_b200 as jt
from oracle import cache as oc

pytestmark = pytest.mark.gpu

BF16, FP16 = torch.bfloat16, torch.float16
BAD_CHUNK = 7


@pytest.fixture(scope="module", autouse=True)
def cuda_ready():
    assert torch.cuda.is_available(), "needs a GPU"
    jt.lib()


def f64(t):
    return t.detach().double().cpu().numpy()


class Batch:
    """Sequences (past, new) with their pages in random order, the pages filled
    with `fill` where no sequence holds a position."""

    def __init__(self, seqs, Hq, Hkv, D, page, dtype, head_major=True, seed=0, fill=float("nan"), tail_rows=0,
                 extra_pages=2):
        g = torch.Generator().manual_seed(seed)
        self.seqs, self.Hq, self.Hkv, self.D, self.page, self.dtype = seqs, Hq, Hkv, D, page, dtype
        B = len(seqs)
        need = [(p + n + page - 1) // page for p, n in seqs]
        n_pages = sum(need) + 3
        order = torch.randperm(n_pages, generator=g).tolist()
        self.table = torch.full((B, max(need + [0]) + extra_pages), 2 ** 31 - 1, dtype=torch.int32)
        shape = (n_pages, Hkv, page, D) if head_major else (n_pages, page, Hkv, D)
        k, v = (torch.full(shape, fill, dtype=dtype) for _ in range(2))
        if head_major:
            k, v = k.transpose(1, 2), v.transpose(1, 2)
        self.k_seq, self.v_seq = [], []
        for b, (p, n) in enumerate(seqs):
            for i in range(need[b]):
                self.table[b, i] = order.pop()
            ks = torch.randn(p + n, Hkv, D, generator=g).to(dtype)
            vs = torch.randn(p + n, Hkv, D, generator=g).to(dtype)
            for t in range(0, p + n, page):
                m = min(page, p + n - t)
                k[self.table[b, t // page], :m] = ks[t:t + m]
                v[self.table[b, t // page], :m] = vs[t:t + m]
            self.k_seq.append(ks)
            self.v_seq.append(vs)
        self.T = sum(n for _, n in seqs) + tail_rows
        self.rows = torch.tensor([sum(n for _, n in seqs[:b]) for b in range(B + 1)], dtype=torch.int32)
        self.past = torch.tensor([p for p, _ in seqs], dtype=torch.int32)
        self.q = torch.randn(self.T, Hq, D, generator=g).to(dtype)
        self.k, self.v = k.cuda(), v.cuda()
        if head_major:  # .cuda() of a transposed view keeps its strides
            assert self.k.stride(1) == D
        self.cache = jt.hia_cache(self.k, self.v)
        self.chunk = jt.hia_cache_chunk(self.table.cuda(), self.past.cuda(), self.rows.cuda())

    def check(self, o, lse, bound=None, scale=None):
        o, lse = f64(o), f64(lse)
        u = torch.finfo(self.dtype).eps / 2
        for b, (p, n) in enumerate(self.seqs):
            r = int(self.rows[b])
            last = np.arange(p, p + n) if bound is None else bound[r:r + n].numpy()
            ro, rl, ra = oc.attend(f64(self.q[r:r + n]), f64(self.k_seq[b]), f64(self.v_seq[b]), last,
                                   self.D ** -0.5 if scale is None else scale)
            assert np.all(np.isfinite(o[r:r + n]))
            tol = u * (ra + np.abs(ro)) * 1.01 + 4e-4 * ra + 1e-7
            err = np.abs(o[r:r + n] - ro)
            assert np.all(err <= tol), f"sequence {b}: {(err - tol).max():.3e} over, error {err.max():.3e}"
            gl = lse[:, r:r + n]
            empty = np.isinf(rl)
            assert np.array_equal(np.isinf(gl), empty) and np.all(gl[empty] == -np.inf)
            assert np.all(np.abs(gl[~empty] - rl[~empty]) <= 2.1e-4 + 1e-6 * np.abs(rl[~empty]))
            assert np.all(o[r:r + n][empty.T] == 0)


def attend(bt, bound=None, **kw):
    o, lse = jt.hia_attn_cache_fwd(bt.cache, bt.chunk, bt.q.cuda(), bound=None if bound is None else bound.cuda(), **kw)
    torch.cuda.synchronize()
    assert jt.hia_get_device_status() == 0
    return o, lse


ROWS = [  # single tokens and few rows: seqs, Hq, Hkv, D, page
    ([(0, 1)], 4, 1, 64, 16),
    ([(1023, 1)], 8, 2, 128, 64),
    ([(15, 1), (16, 1), (17, 1), (0, 1), (127, 1), (128, 1)], 4, 2, 64, 16),
    ([(300, 1), (0, 0), (77, 3), (5, 0), (1000, 2)], 4, 4, 128, 32),    # g = 1, sequences without new tokens
    ([(700, 1), (3, 1), (255, 1)], 7, 1, 128, 256),                      # g = 7
    ([(900, 1)] * 3, 16, 1, 64, 128),                                    # one full row tile
    ([(2500, 1), (40, 1)], 8, 8, 128, 64),
    ([(6000, 1)], 4, 1, 128, 64),                                        # split over the keys
    ([(10, 4), (400, 1), (90, 2)], 8, 2, 64, 64),
]
TILES = [  # many rows
    ([(0, 1)], 128, 1, 64, 16),                                          # the largest group
    ([(0, 129)], 4, 1, 64, 16),
    ([(1000, 70), (3, 1), (0, 200), (64, 64)], 8, 2, 128, 64),
    ([(513, 100), (0, 0), (1, 33)], 6, 2, 128, 128),                     # g = 3: 126 of 128 rows
    ([(0, 260)], 5, 5, 64, 256),                                         # g = 1
    ([(37, 90)], 7, 1, 128, 32),
    ([(2000, 20)], 32, 2, 128, 64),                                      # g = 16, split over the keys
    ([(100, 3), (5000, 40), (0, 17)], 8, 1, 64, 16),
    ([(127, 1), (128, 300), (129, 2)], 40, 1, 64, 32),                   # g = 40: 3 tokens a tile
]


@pytest.mark.parametrize("seqs,Hq,Hkv,D,page", ROWS + TILES)
@pytest.mark.parametrize("dtype,head_major", [(BF16, True), (FP16, False)])
def test_causal(seqs, Hq, Hkv, D, page, dtype, head_major):
    """Slots that no position holds are NaN, unused table entries are no pages."""
    bt = Batch(seqs, Hq, Hkv, D, page, dtype, head_major)
    bt.check(*attend(bt))


@pytest.mark.parametrize("seqs,Hq,Hkv,D,page", ROWS[2:5] + ROWS[7:] + TILES[1:8])
def test_row_bounds(seqs, Hq, Hkv, D, page):
    """Random last visible positions, below and past the sequence, and rows
    that see nothing."""
    bt = Batch(seqs, Hq, Hkv, D, page, BF16, seed=3)
    g = torch.Generator().manual_seed(4)
    bound = torch.cat([torch.randint(-2, max(p + n + 3, 1), (n,), generator=g) for p, n in seqs]).int()
    bound[::5] = -1
    bt.check(*attend(bt, bound), bound=bound)


def test_all_rows_empty():
    bt = Batch([(50, 3), (0, 200)], 4, 1, 64, 16, BF16)
    for seqs in ([(50, 3), (0, 200)], [(500, 1), (20, 2)]):
        bt = Batch(seqs, 4, 1, 64, 16, BF16)
        o, lse = attend(bt, torch.full((bt.T,), -7, dtype=torch.int32))
        assert torch.all(o == 0) and torch.all(lse == -float("inf"))


@pytest.mark.parametrize("what", ["v", "k"])
@pytest.mark.parametrize("seqs,Hq,Hkv,D,page", [
    ([(30, 3), (250, 4)], 4, 1, 64, 16), ([(3000, 2), (100, 4)], 8, 2, 128, 64),      # rows kernel
    ([(200, 20), (60, 90), (0, 300)], 4, 1, 64, 16), ([(4000, 20)], 8, 1, 128, 64),   # tiles kernel, one and two row tiles
    ([(100, 33), (0, 70), (37, 200)], 8, 2, 128, 32),
])
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("bounded", [False, True])
def test_infinities_and_nan_in_keys_and_values(what, seqs, Hq, Hkv, D, page, dtype, bounded):
    """New tokens' keys or values hold infinities and NaN: rows that do not see
    them are as if they were not there, rows that do have them by the formula
    (a NaN key makes the row NaN; an infinite value an infinite element)."""
    bt = Batch(seqs, Hq, Hkv, D, page, dtype, seed=5)
    g = torch.Generator().manual_seed(6)
    bad = [float("nan")] if what == "k" else [float("nan"), float("inf"), -float("inf")]
    for b, (p, n) in enumerate(seqs):
        for i in range(3):
            t = p + int(torch.randint(n // 2, n, (1,), generator=g))
            h, d = int(torch.randint(Hkv, (1,), generator=g)), int(torch.randint(D, (1,), generator=g))
            x = bad[i % len(bad)]
            (bt.k_seq if what == "k" else bt.v_seq)[b][t, h, d] = x
            (bt.k if what == "k" else bt.v)[int(bt.table[b, t // page]), t % page, h, d] = x
    bound = None
    if bounded:
        bound = torch.cat([torch.randint(0, p + n, (n,), generator=g) for p, n in seqs]).int()
        bound[::7] = -1
    o, lse = attend(bt, bound)
    o, lse = f64(o), f64(lse)
    u = torch.finfo(dtype).eps / 2
    n_odd = 0
    for b, (p, n) in enumerate(seqs):
        r = int(bt.rows[b])
        last = np.arange(p, p + n) if bound is None else bound[r:r + n].numpy()
        with np.errstate(invalid="ignore"):
            ro, rl, ra = oc.attend(f64(bt.q[r:r + n]), f64(bt.k_seq[b]), f64(bt.v_seq[b]), last, D ** -0.5)
        go, gl = o[r:r + n], lse[:, r:r + n]
        assert np.array_equal(np.isnan(go), np.isnan(ro))
        inf = np.isinf(ro)
        assert np.array_equal(np.isinf(go), inf) and np.array_equal(go[inf], ro[inf])
        fin = np.isfinite(ro)
        n_odd += np.count_nonzero(~fin)
        assert np.all(np.abs(go[fin] - ro[fin]) <= (u * (ra + np.abs(ro)) * 1.01 + 4e-4 * ra + 1e-7)[fin])
        assert np.array_equal(np.isnan(gl), np.isnan(rl)) and np.array_equal(np.isinf(gl), np.isinf(rl))
        fin = np.isfinite(rl)
        assert np.all(np.abs(gl[fin] - rl[fin]) <= 2.1e-4 + 1e-6 * np.abs(rl[fin]))
    assert n_odd > 0 or bounded


@pytest.mark.parametrize("seqs", [[(200, 300)], [(1000, 4)]])
def test_image_span(seqs):
    """The image rows of a chunk see each other, its text rows are causal."""
    bt = Batch(seqs, 4, 1, 128, 64, BF16)
    p, n = seqs[0]
    bound = torch.arange(p, p + n, dtype=torch.int32)
    bound[1:n - 1] = p + n - 2
    bt.check(*attend(bt, bound), bound=bound)


@pytest.mark.parametrize("scale", [1.0, 3.0, 1e-3])
@pytest.mark.parametrize("seqs", [[(700, 1)], [(400, 150)]])
def test_scales(scale, seqs):
    """Large scores move the running maximum (the output is rescaled); the
    scores' fp32 error scales with `scale`: queries are scaled down with it."""
    bt = Batch(seqs, 4, 1, 64, 16, FP16, seed=9)
    bt.q *= 2.0 ** -2 if scale > 1 else 1.0
    # scale D 2^-23 sum|qk|, sum|qk| <= 70 |q| at D = 64: at most 1.6e-3 at scale 3
    o, lse = attend(bt, scale=scale)
    o, lse = f64(o), f64(lse)
    p, n = seqs[0]
    ro, rl, ra = oc.attend(f64(bt.q), f64(bt.k_seq[0]), f64(bt.v_seq[0]), np.arange(p, p + n), scale)
    u = 2.0 ** -11
    assert np.all(np.abs(o - ro) <= u * (ra + np.abs(ro)) * 1.01 + 4e-3 * ra + 1e-7)
    assert np.all(np.abs(lse - rl) <= 2e-3 + 1e-6 * np.abs(rl))


def test_scores_growing_along_the_keys():
    """Each 128-key tile's scores above the last one's by more than the lazy
    rescale's threshold, and one far below: the running maximum moves often."""
    for seqs in ([(1500, 1)], [(1200, 130)]):
        bt = Batch(seqs, 4, 1, 64, 16, FP16, seed=2)
        L = sum(seqs[0])
        step = torch.arange(L) // 128
        boost = torch.where(step % 3 == 2, -step.float(), step.float())
        ks = (bt.k_seq[0].float() * 0.05)
        ks[:, :, 0] = boost[:, None] * 2
        ks = ks.half()
        bt.k_seq[0] = ks
        for t in range(0, L, 16):
            m = min(16, L - t)
            bt.k[bt.table[0, t // 16], :m] = ks[t:t + m].cuda()
        bt.q[:, :, 0] = 40.0
        # scores up to 40 * 22 / 8 = 110: fp32 products of 880 within 880 * 2^-23 * 64 / 8 = 8.4e-4 each
        o, lse = attend(bt)
        p, n = seqs[0]
        ro, rl, ra = oc.attend(f64(bt.q), f64(ks), f64(bt.v_seq[0]), np.arange(p, p + n), 0.125)
        assert np.all(np.abs(f64(o) - ro) <= 2.0 ** -11 * (ra + np.abs(ro)) * 1.01 + 2e-3 * ra + 1e-7)
        assert np.all(np.abs(f64(lse) - rl) <= 1.1e-3 + 1e-6 * np.abs(rl))


@pytest.mark.parametrize("seqs", [[(0, 1), (40, 1), (700, 1)], [(0, 150), (1, 17), (500, 90)]])
@pytest.mark.parametrize("level", [-300.0, 300.0])
@pytest.mark.parametrize("D", [64, 128])
def test_scores_far_from_zero(seqs, level, D):
    """Every score of every row near -300 or 300 (unit columns added to small
    random ones): the maximum is the row's own, over visible keys alone; slots
    that hold nothing are at 3e38."""
    bt = Batch(seqs, 4, 1, D, 16, BF16, fill=3e38)
    bt.q[:] = (bt.q.float() * 0.125).to(BF16)
    bt.q[:, :, 0] = 32.0
    far = level * D ** 0.5 / 32.0  # a multiple of 1/8 below 128: exact in bf16
    far = round(far) * 1.0
    for b, (p, n) in enumerate(bt.seqs):
        bt.k_seq[b][:, :, 0] = far
        for t in range(p + n):
            bt.k[bt.table[b, t // bt.page], t % bt.page, :, 0] = far
    o, lse = attend(bt)
    # scores: one product of 32 |far| <= 32 * 107 beside D small ones (sum of
    # magnitudes <= 32): fp32 sums within 3460 * 2^-23 * D / sqrt(D) <= 4.7e-3,
    # in their exponentials' numerator and sum: 9.4e-3 a; the scaled score in
    # log2 units (below 512) is rounded twice more, 2 * 2^-15 each
    for b, (p, n) in enumerate(bt.seqs):
        r = int(bt.rows[b])
        ro, rl, ra = oc.attend(f64(bt.q[r:r + n]), f64(bt.k_seq[b]), f64(bt.v_seq[b]), np.arange(p, p + n), D ** -0.5)
        assert np.all(np.abs(f64(o[r:r + n]) - ro) <= 2.0 ** -8 * (ra + np.abs(ro)) * 1.01 + 1e-2 * ra)
        assert np.all(np.abs(f64(lse[:, r:r + n]) - rl) <= 5e-3)


@pytest.mark.parametrize("seqs,Hq,Hkv", [([(70, 1), (300, 1)], 8, 2), ([(70, 90), (3, 40)], 8, 2)])
def test_strides_and_rows_behind_the_last_sequence(seqs, Hq, Hkv):
    """q a view of a fused projection, o a view of a wider tensor; rows behind
    the last sequence are left as they were."""
    D = 64
    bt = Batch(seqs, Hq, Hkv, D, 16, BF16, tail_rows=9)
    g = Hq // Hkv
    fused = torch.full((bt.T, Hkv, g + 2, D), float("nan"), dtype=BF16, device="cuda")
    fused[:, :, :g] = bt.q.cuda().reshape(bt.T, Hkv, g, D)
    wide = torch.full((bt.T, Hkv, g + 1, D), 5.0, dtype=BF16, device="cuda")
    lse = torch.full((Hq, bt.T), 9.0, device="cuda")
    jt.hia_attn_cache_fwd(bt.cache, bt.chunk, fused[:, :, :g], o=wide[:, :, :g], lse=lse)
    o, want_lse = attend(bt, o=torch.full((bt.T, Hq, D), 5.0, dtype=BF16, device="cuda"),
                         lse=torch.full((Hq, bt.T), 9.0, device="cuda"))
    assert torch.equal(wide[:, :, :g].reshape(bt.T, Hq, D), o) and torch.equal(lse, want_lse)
    assert torch.all(wide[:, :, g] == 5.0)
    assert torch.all(o[-9:] == 5.0) and torch.all(lse[:, -9:] == 9.0)
    bt.check(o, lse)


def test_shared_prefix_pages():
    """Two sequences reading the same pages."""
    bt = Batch([(128, 1), (128, 1)], 4, 1, 64, 32, BF16, fill=0.0)
    bt.table[1, :4] = bt.table[0, :4]
    bt.k_seq[1] = torch.cat([bt.k_seq[0][:128], bt.k_seq[1][128:]])
    bt.v_seq[1] = torch.cat([bt.v_seq[0][:128], bt.v_seq[1][128:]])
    bt.chunk = jt.hia_cache_chunk(bt.table.cuda(), bt.past.cuda(), bt.rows.cuda())
    bt.check(*attend(bt))


@pytest.mark.parametrize("seqs", [[(4000, 1)], [(4000, 30), (100, 20)], [(777, 1)] * 40])
def test_repeatable(seqs):
    bt = Batch(seqs, 8, 2, 128, 64, BF16)
    a = attend(bt)
    for _ in range(3):
        b = attend(bt)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_more_sequences_than_threads():
    """More sequences than a block has threads, most without new tokens."""
    seqs = [(i % 50, 1 if i % 7 == 3 else 0) for i in range(900)]
    bt = Batch(seqs, 4, 1, 64, 16, BF16)
    bt.check(*attend(bt))
    seqs = [(i % 50, 30 if i % 97 == 3 else 0) for i in range(900)]
    bt = Batch(seqs, 4, 1, 64, 16, BF16)
    bt.check(*attend(bt))


@pytest.mark.parametrize("seqs", [[(500, 1), (60, 1)], [(100, 90), (7, 50)]])
def test_bad_chunks_are_reported(seqs):
    """Pages and lengths that do not fit: reported, the sequence skipped (or
    the page read as zeros), the other sequence's rows right."""
    def run(edit):
        bt = Batch(seqs, 4, 1, 64, 16, BF16)
        edit(bt)
        bt.chunk = jt.hia_cache_chunk(bt.table.cuda(), bt.past.cuda(), bt.rows.cuda())
        o = torch.full((bt.T, 4, 64), 5.0, dtype=BF16, device="cuda")
        lse = torch.full((4, bt.T), 5.0, device="cuda")
        jt.hia_attn_cache_fwd(bt.cache, bt.chunk, bt.q.cuda(), o=o, lse=lse)
        torch.cuda.synchronize()
        assert jt.hia_get_device_status() == BAD_CHUNK
        assert jt.hia_get_device_status() == 0
        return bt, o, lse

    n0 = seqs[0][1]

    def other_right(bt, o, lse):
        keep = bt.seqs
        bt.seqs = [(0, 0), seqs[1]]
        bt.rows[0] = n0
        bt.check(o, lse)
        bt.seqs = keep

    def page(bt, x):
        bt.table[0, 2] = x
    for x in (-1, -2 ** 31, 2 ** 31 - 1, 10 ** 6):
        other_right(*run(lambda bt: page(bt, x)))

    def past(bt, x):
        bt.past[0] = x
    for x in (-1, 10 ** 9, 2 ** 31 - 1):
        bt, o, lse = run(lambda bt: past(bt, x))
        assert torch.all(o[:n0] == 5.0) and torch.all(lse[:, :n0] == 5.0)
        bt.past[0] = seqs[0][0]
        other_right(bt, o, lse)

    def rows(bt, i, x):
        bt.rows[i] = x
    bt, o, lse = run(lambda bt: rows(bt, 0, -3))
    assert torch.all(o[:n0] == 5.0)
    run(lambda bt: rows(bt, 2, 10 ** 6))
    run(lambda bt: rows(bt, 1, 10 ** 6))


@pytest.mark.parametrize("head_major", [True, False])
def test_offsets_past_32_bits(head_major):
    """Pages more than 2^31 elements (and 2^32 bytes) into the pool."""
    Hkv, page, D = 8, 64, 128
    n_pages = (1 << 31) // (Hkv * page * D) + 40
    shape = (n_pages, Hkv, page, D) if head_major else (n_pages, page, Hkv, D)
    k, v = torch.empty(shape, dtype=BF16, device="cuda"), torch.empty(shape, dtype=BF16, device="cuda")
    if head_major:
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    cache = jt.hia_cache(k, v)
    g = torch.Generator().manual_seed(0)
    for n in (1, 90):
        past = 150
        L = past + n
        ids = [n_pages - 1, 0, n_pages - 7, n_pages - 2]
        table = torch.tensor([ids], dtype=torch.int32, device="cuda")
        ks, vs = (torch.randn(L, Hkv, D, generator=g).to(BF16) for _ in range(2))
        q = torch.randn(n, 16, D, generator=g).to(BF16)
        for t in range(0, past, page):
            m = min(page, past - t)
            k[ids[t // page], :m] = ks[t:t + m].cuda()
            v[ids[t // page], :m] = vs[t:t + m].cuda()
        chunk = jt.hia_cache_chunk(table, torch.tensor([past], dtype=torch.int32, device="cuda"),
                                   torch.tensor([0, n], dtype=torch.int32, device="cuda"))
        assert jt.hia_cache_append(cache, chunk, None, ks[past:].cuda(), vs[past:].cuda()) is None
        o, lse = jt.hia_attn_cache_fwd(cache, chunk, q.cuda())
        torch.cuda.synchronize()
        assert jt.hia_get_device_status() == 0
        ro, rl, ra = oc.attend(f64(q), f64(ks), f64(vs), np.arange(past, L), D ** -0.5)
        assert np.all(np.abs(f64(o) - ro) <= 2.0 ** -8 * (ra + np.abs(ro)) * 1.01 + 4e-4 * ra)
        assert np.all(np.abs(f64(lse) - rl) <= 2.1e-4 + 1e-6 * np.abs(rl))


# ---------------------------------------------------------------- append
APPEND = [  # seqs, Hq, Hkv, D, page, axes, sections
    ([(0, 1)], 4, 1, 64, 16, 1, None),
    ([(15, 1), (16, 1), (0, 1), (31, 2)], 8, 2, 128, 16, 2, None),
    ([(1000, 70), (3, 0), (0, 200), (63, 64)], 6, 2, 128, 64, 3, [16, 24, 24]),
    ([(100, 1)] * 70, 32, 8, 128, 256, 2, None),
    ([(5, 300)], 5, 5, 64, 32, 2, None),
]


@pytest.mark.parametrize("seqs,Hq,Hkv,D,page,axes,sections", APPEND)
@pytest.mark.parametrize("dtype,head_major,norm,turn", [(BF16, True, True, True), (FP16, False, False, True),
                                                        (BF16, False, True, False), (FP16, True, False, False)])
def test_append(seqs, Hq, Hkv, D, page, axes, sections, dtype, head_major, norm, turn):
    bt = Batch(seqs, Hq, Hkv, D, page, dtype, head_major, fill=3.0, tail_rows=5)
    g = Hq // Hkv
    gen = torch.Generator().manual_seed(1)
    T = bt.T
    fused = torch.randn(T, Hkv, g + 2, D, generator=gen).to(dtype)
    pos = torch.randint(0, 9000, (T, axes), generator=gen, dtype=torch.int32)
    wq, wk = (1 + 0.1 * torch.randn(D, generator=gen) for _ in range(2))
    k0, v0 = bt.k.clone(), bt.v.clone()
    d = fused.cuda()
    q_out = torch.full((T, Hq, D), 5.0, dtype=dtype, device="cuda")
    jt.hia_cache_append(bt.cache, bt.chunk, d[:, :, :g], d[:, :, g], d[:, :, g + 1],
                        plan=jt.hia_rope_plan(D, axes, sections=sections) if turn else None,
                        pos=pos.cuda() if turn else None, qk_norm=(wq.cuda(), wk.cuda(), 1e-5) if norm else None,
                        q_out=q_out)
    torch.cuda.synchronize()
    assert jt.hia_get_device_status() == 0
    pairs = oc.rope_pairs(D, axes, sections, 10000.0, False)
    fi = torch.finfo(dtype)
    n_rows = int(bt.rows[-1])

    def expect(x, w):
        y = oc.rotate(x, pos.numpy(), pairs) if turn else x
        mag = np.abs(x[..., :D // 2]) + np.abs(x[..., D // 2:])
        mag = 1.01e-6 * np.concatenate([mag, mag], -1) if turn else 0.0
        if norm:
            r = 1 / np.sqrt((y * y).mean(-1, keepdims=True) + 1e-5)
            y, mag = w * y * r, np.abs(w) * r * (mag + 2e-6 * np.abs(y))  # r, and three products, within 2e-6
        return y, fi.eps / 2 * np.abs(y) + mag + fi.smallest_normal * fi.eps / 2

    yq, tq = expect(f64(fused[:, :, :g].reshape(T, Hq, D)), f64(wq))
    yk, tk = expect(f64(fused[:, :, g]), f64(wk))
    got = f64(q_out)
    assert np.all(np.abs(got - yq)[:n_rows] <= tq[:n_rows])
    assert np.all(got[n_rows:] == 5.0), "rows behind the last sequence"
    kk, vv = bt.k.clone(), bt.v.clone()
    for b, (p, n) in enumerate(seqs):
        for i in range(n):
            t, r = p + i, int(bt.rows[b]) + i
            pg, sl = int(bt.table[b, t // page]), t % page
            assert np.all(np.abs(f64(kk[pg, sl]) - yk[r]) <= tk[r])
            assert torch.equal(vv[pg, sl].cpu(), fused[r, :, g + 1])
            kk[pg, sl] = k0[pg, sl]
            vv[pg, sl] = v0[pg, sl]
    assert torch.equal(kk, k0) and torch.equal(vv, v0), "other slots are left as they were"


def test_append_in_place_and_keys_only():
    bt = Batch([(30, 40), (0, 7)], 8, 2, 64, 16, BF16, fill=0.0)
    q, k, v = (torch.randn(bt.T, h, 64, generator=torch.Generator().manual_seed(h)).to(BF16).cuda() for h in (8, 2, 3))
    v = v[:, :2]
    plan, pos = jt.hia_rope_plan(64, 1), torch.arange(bt.T, dtype=torch.int32, device="cuda")[:, None]
    a = jt.hia_cache_append(bt.cache, bt.chunk, q, k, v, plan=plan, pos=pos)
    k1, v1 = bt.k.clone(), bt.v.clone()
    bt.k.zero_(), bt.v.zero_()
    q2 = q.clone()
    assert jt.hia_cache_append(bt.cache, bt.chunk, q2, k, v, plan=plan, pos=pos, q_out=q2) is q2
    assert torch.equal(q2, a) and torch.equal(
        torch.where(bt.k != 0, bt.k, k1), k1)
    bt.k.copy_(k1), bt.v.copy_(v1)
    assert jt.hia_cache_append(bt.cache, bt.chunk, None, k, v, plan=plan, pos=pos) is None
    assert torch.equal(bt.k, k1) and torch.equal(bt.v, v1)


def test_append_reports_bad_chunks():
    def run(edit):
        bt = Batch([(20, 30), (40, 1)], 4, 1, 64, 16, BF16, fill=0.0)
        k0 = bt.k.clone()
        edit(bt)
        chunk = jt.hia_cache_chunk(bt.table.cuda(), bt.past.cuda(), bt.rows.cuda())
        x = torch.ones(bt.T, 1, 64, dtype=BF16, device="cuda")
        q = torch.ones(bt.T, 4, 64, dtype=BF16, device="cuda")
        out = torch.full_like(q, 5.0)
        jt.hia_cache_append(bt.cache, chunk, q, x, x, q_out=out)
        torch.cuda.synchronize()
        assert jt.hia_get_device_status() == BAD_CHUNK
        return bt, k0, out

    def page(bt):
        bt.table[0, 2] = 1000
    bt, k0, out = run(page)
    assert torch.all(out == 1.0)
    pg = bt.table[0].tolist()
    assert torch.all(bt.k[pg[1], 4:] == 1.0) and torch.all(bt.k[pg[3], :2] == 1.0)

    def past(bt):
        bt.past[0] = -5
    bt, k0, out = run(past)
    assert torch.all(out[:30] == 5.0) and torch.all(out[30:] == 1.0)
    assert torch.all(bt.k[int(bt.table[1, 2]), 8] == 1.0)

    def long(bt):
        bt.past[0] = 10 ** 6
    run(long)


# ---------------------------------------------------------------- together
def test_generation_is_the_training_forward():
    """A sample of text, an image and text, generated: the prompt as a chunk,
    the image as a chunk (denoised twice: its rows are appended again over the
    first try), then text token by token.  Every row's output and log-sum-exp
    are those of the whole sequence at once (hia_attn_fwd with the same 2D RoPE
    and QK norm), and of its oracle within the tolerances above plus those of
    the forward."""
    P, h, w, sfx, Hq, Hkv, D = 140, 12, 16, 9, 8, 2, 128
    L = P + h * w + sfx
    gen = torch.Generator().manual_seed(11)
    qkv = torch.randn(L, Hkv, Hq // Hkv + 2, D, generator=gen).to(BF16).cuda()
    wq, wk = (1 + 0.1 * torch.randn(D, generator=gen).cuda() for _ in range(2))
    norm = (wq, wk, 1e-5)
    pos = torch.tensor([[P + (n - P) % w, P + (n - P) // w] if P <= n < P + h * w else [n, n] for n in range(L)],
                       dtype=torch.int32, device="cuda")
    plan = jt.hia_rope_plan(D, 2)
    page = 32
    n_pages = (L + page - 1) // page
    pages = [torch.full((n_pages, Hkv, page, D), float("nan"), dtype=BF16, device="cuda").transpose(1, 2)
             for _ in range(2)]
    cache = jt.hia_cache(*pages)
    table = torch.randperm(n_pages, generator=gen).int()[None].cuda()
    o = torch.empty(L, Hq, D, dtype=BF16, device="cuda")
    lse = torch.empty(Hq, L, device="cuda")

    def step(a, b, x, image=False):
        n = b - a
        chunk = jt.hia_cache_chunk(table, torch.tensor([a], dtype=torch.int32, device="cuda"),
                                   torch.tensor([0, n], dtype=torch.int32, device="cuda"))
        q = jt.hia_cache_append(cache, chunk, x[:, :, :-2], x[:, :, -2], x[:, :, -1], plan=plan, pos=pos[a:b],
                                qk_norm=norm)
        bound = torch.full((n,), b - 1, dtype=torch.int32, device="cuda") if image else None
        return jt.hia_attn_cache_fwd(cache, chunk, q, bound=bound)

    def keep(a, b, r):
        o[a:b], lse[:, a:b] = r

    keep(0, 100, step(0, 100, qkv[:100]))
    keep(100, P, step(100, P, qkv[100:P]))
    step(P, P + h * w, qkv[P:P + h * w].flip(0).contiguous(), image=True)  # a noisier image
    keep(P, P + h * w, step(P, P + h * w, qkv[P:P + h * w], image=True))
    for t in range(P + h * w, L):
        keep(t, t + 1, step(t, t + 1, qkv[t:t + 1]))
    torch.cuda.synchronize()
    assert jt.hia_get_device_status() == 0
    seg = jt.hia_segments_build([(P, h, w, sfx)], L)
    c, s = jt.hia_rope2d_tables(seg, D)
    x = qkv[None]
    fo, flse = jt.hia_attn_fwd(seg, x[:, :, :, :-2], x[:, :, :, -2], x[:, :, :, -1], c, s, qk_norm=norm)
    torch.cuda.synchronize()
    # both within the attention tolerance of the same exact result, given the
    # same rotated rows (which may differ by a bf16 step where fp32 rounds apart)
    rel = (o.float() - fo[0].float()).norm() / fo.float().norm()
    assert rel <= 2 ** -7
    assert (o.float() - fo[0].float()).abs().max() <= 2e-2
    assert (lse - flse[0]).abs().max() <= 1e-2 and (lse - flse[0]).abs().mean() <= 1e-3


def test_captured_step_sees_new_lengths():
    """One captured decode step (append + attention), replayed as the sequences
    grow: lengths and positions are read on the device."""
    B, Hq, Hkv, D, page = 3, 8, 2, 64, 16
    start, steps = [0, 15, 300], 20
    seqs = [(p, steps) for p in start]
    bt = Batch(seqs, Hq, Hkv, D, page, BF16, fill=float("nan"))
    for b, p in enumerate(start):  # the cache holds the past only
        for t in range(p, p + steps):
            bt.k[bt.table[b, t // page], t % page] = float("nan")
            bt.v[bt.table[b, t // page], t % page] = float("nan")
    past = torch.tensor(start, dtype=torch.int32, device="cuda")
    rows = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    chunk = jt.hia_cache_chunk(bt.table.cuda(), past, rows)
    q, k, v = (torch.zeros(B, h, D, dtype=BF16, device="cuda") for h in (Hq, Hkv, Hkv))
    qo, o = torch.zeros_like(q), torch.zeros_like(q)
    lse = torch.zeros(Hq, B, device="cuda")
    ws = torch.zeros(jt.hia_attn_cache_workspace_bytes(bt.cache, chunk, B, Hq), dtype=torch.uint8, device="cuda")

    def step():
        jt.hia_cache_append(bt.cache, chunk, q, k, v, q_out=qo)
        jt.hia_attn_cache_fwd(bt.cache, chunk, qo, o=o, lse=lse, workspace=ws)

    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    for i in range(steps):
        for b in range(B):
            q[b] = bt.q[b * steps + i].cuda()
            k[b] = bt.k_seq[b][start[b] + i].cuda()
            v[b] = bt.v_seq[b][start[b] + i].cuda()
        past.copy_(torch.tensor([p + i for p in start]))
        graph.replay()
        torch.cuda.synchronize()
        assert jt.hia_get_device_status() == 0
        for b, p in enumerate(start):
            ro, rl, ra = oc.attend(f64(bt.q[b * steps + i:b * steps + i + 1]), f64(bt.k_seq[b][:p + i + 1]),
                                   f64(bt.v_seq[b][:p + i + 1]), [p + i], D ** -0.5)
            assert np.all(np.abs(f64(o[b]) - ro[0]) <= 2.0 ** -8 * (ra[0] + np.abs(ro[0])) * 1.01 + 4e-4 * ra[0])
            assert np.all(np.abs(f64(lse[:, b]) - rl[:, 0]) <= 2.1e-4 + 1e-6 * np.abs(rl[:, 0]))


def test_two_streams_at_once():
    """Two batches on two streams, each with its own workspace."""
    a = Batch([(3000, 1), (50, 1)], 8, 2, 128, 64, BF16, seed=1)
    b = Batch([(900, 60), (4, 90)], 8, 2, 128, 64, BF16, seed=2)
    want = [attend(x) for x in (a, b)]
    qa, qb = a.q.cuda(), b.q.cuda()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        with torch.cuda.stream(sa):
            ra = jt.hia_attn_cache_fwd(a.cache, a.chunk, qa)
        with torch.cuda.stream(sb):
            rb = jt.hia_attn_cache_fwd(b.cache, b.chunk, qb)
        torch.cuda.synchronize()
        for got, ref in ((ra, want[0]), (rb, want[1])):
            assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


def test_two_graphs_share_a_workspace():
    """A decode step and a prompt step captured with one workspace and
    replayed in turn: nothing of a call outlasts it."""
    a = Batch([(3000, 1), (50, 1), (700, 1)], 8, 2, 128, 64, BF16, seed=1)
    b = Batch([(2500, 60), (4, 90)], 8, 2, 128, 64, BF16, seed=2)
    want = [attend(x) for x in (a, b)]
    ws = torch.full((max(jt.hia_attn_cache_workspace_bytes(x.cache, x.chunk, x.T, x.Hq) for x in (a, b)),), 0xff,
                    dtype=torch.uint8, device="cuda")
    graphs, outs, qs = [], [], [x.q.cuda() for x in (a, b)]
    torch.cuda.synchronize()
    for x, q in zip((a, b), qs):
        o, lse = torch.zeros_like(q), torch.zeros(x.Hq, x.T, device="cuda")
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            jt.hia_attn_cache_fwd(x.cache, x.chunk, q, o=o, lse=lse, workspace=ws)
        outs.append((o, lse))
    for _ in range(4):
        for graph, got, ref in zip(graphs, outs, want):
            got[0].fill_(3.0)
            got[1].fill_(3.0)
            graph.replay()
            assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    assert jt.hia_get_device_status() == 0


@pytest.mark.parametrize("seqs,Hq,Hkv", [([(70, 1), (300, 1)], 3, 3), ([(70, 1), (300, 1)], 4, 1),
                                         ([(70, 90), (3, 40)], 3, 3), ([(70, 90), (3, 40)], 6, 1), ([(600, 1)], 2, 2),
                                         ([(0, 1)], 17, 1)])
@pytest.mark.parametrize("pad", [8, 16, 24])
def test_outputs_off_the_widest_alignment(seqs, Hq, Hkv, pad):
    """Rows that begin 16, 32 or 48 bytes apart from a multiple of the widest
    store; one head a group, one kv head, one row."""
    D = 64
    bt = Batch(seqs, Hq, Hkv, D, 16, BF16)
    want, want_lse = attend(bt)
    flat_o = torch.full((bt.T * (Hq * D + pad) + 64,), 5.0, dtype=BF16, device="cuda")
    flat_q = torch.full_like(flat_o, float("nan"))
    o, q = (x[pad:].as_strided((bt.T, Hq, D), (Hq * D + pad, D, 1)) for x in (flat_o, flat_q))
    q.copy_(bt.q)
    _, lse = jt.hia_attn_cache_fwd(bt.cache, bt.chunk, q, o=o)
    assert torch.equal(o, want) and torch.equal(lse, want_lse)
    keep = torch.ones_like(flat_o, dtype=torch.bool)
    keep[pad:].as_strided((bt.T, Hq, D), (Hq * D + pad, D, 1)).fill_(False)
    assert torch.all(flat_o[keep] == 5.0)


def test_append_one_row_for_all():
    """Inputs with a row stride of 0."""
    seqs, D = [(7, 5), (3, 40)], 64
    bt = Batch(seqs, 8, 2, D, 16, BF16)
    q, kv = bt.q[:1].cuda(), torch.randn(1, 2, D, generator=torch.Generator().manual_seed(9)).to(BF16).cuda()
    pos = torch.arange(2 * bt.T, dtype=torch.int32, device="cuda").view(bt.T, 2)
    plan, got = jt.hia_rope_plan(D, 2), []
    for rows in (lambda x: x.expand(bt.T, -1, -1), lambda x: x.expand(bt.T, -1, -1).contiguous()):
        qo = jt.hia_cache_append(bt.cache, bt.chunk, rows(q), rows(kv), rows(kv), plan=plan, pos=pos)
        got.append((qo, bt.k.clone(), bt.v.clone()))
    for a, b in zip(*got):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("tail", [4, 300])
def test_no_sequence_has_new_tokens(tail):
    bt = Batch([(5, 0), (40, 0)], 8, 2, 64, 16, BF16, tail_rows=tail)
    o, lse = (torch.full(s, 5.0, dtype=t, device="cuda") for s, t in (((bt.T, 8, 64), BF16), ((8, bt.T), torch.float32)))
    attend(bt, o=o, lse=lse)
    assert torch.all(o == 5.0) and torch.all(lse == 5.0)


def test_refused_tensors():
    bt = Batch([(5, 3)], 4, 1, 64, 16, BF16)
    q, x = bt.q.cuda(), torch.zeros(3, 1, 64, dtype=BF16, device="cuda")
    n = jt.hia_attn_cache_workspace_bytes(bt.cache, bt.chunk, 3, 4)
    with pytest.raises(ValueError):
        jt.hia_attn_cache_fwd(bt.cache, bt.chunk, q, workspace=torch.empty(n, dtype=torch.uint8))  # on the host
    with pytest.raises(ValueError):
        jt.hia_attn_cache_fwd(bt.cache, bt.chunk, q, workspace=torch.empty(n - 1, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        jt.hia_attn_cache_fwd(bt.cache, bt.chunk, q, workspace=torch.empty(n, 2, dtype=torch.uint8, device="cuda")[:, 0])
    with pytest.raises(ValueError):
        jt.hia_attn_cache_fwd(bt.cache, bt.chunk, q.half())
    with pytest.raises(ValueError):
        jt.hia_cache_append(bt.cache, bt.chunk, q, x, x, qk_norm=(torch.ones(64), torch.ones(64), 1e-5))
    table, past, rows = bt.chunk.pages, bt.chunk.past, bt.chunk.rows
    with pytest.raises(ValueError):
        jt.Chunk(table, past.cpu(), rows)
    with pytest.raises(ValueError):
        jt.Cache(bt.k, bt.v.cpu())
    with pytest.raises(jt.HiaError):  # its rows lie on one another
        jt.hia_attn_cache_fwd(bt.cache, bt.chunk, q[:1].expand(3, -1, -1))
    with pytest.raises(jt.HiaError):
        jt.hia_attn_cache_fwd(bt.cache, bt.chunk, q, o=torch.zeros(1, 4, 64, dtype=BF16, device="cuda").expand(3, -1, -1))


def test_nothing_to_do():
    bt = Batch([(5, 3)], 4, 1, 64, 16, BF16)
    q = torch.empty(0, 4, 64, dtype=BF16, device="cuda")
    o, lse = jt.hia_attn_cache_fwd(bt.cache, bt.chunk, q)
    assert o.shape == (0, 4, 64) and lse.shape == (4, 0)
    empty = jt.hia_cache_chunk(*(torch.empty(s, dtype=torch.int32, device="cuda") for s in ((0, 4), (0,), (1,))))
    q = torch.full((3, 4, 64), 2.0, dtype=BF16, device="cuda")
    o = torch.full_like(q, 5.0)
    jt.hia_attn_cache_fwd(bt.cache, empty, q, o=o)
    assert torch.all(o == 5.0)


def test_profile_names():
    bt = Batch([(5, 3)], 4, 1, 64, 16, BF16)
    jt.hia_profile_begin()
    x = torch.zeros(3, 1, 64, dtype=BF16, device="cuda")
    jt.hia_cache_append(bt.cache, bt.chunk, None, x, x)
    attend(bt)
    assert {"cache_append", "attn_cache_rows", "attn_cache_plan"} <= set(jt.hia_profile_end())
