"""GPU tests of the attention over the cache at the ends of its number range:
weights far below a row's largest, infinite keys, values that are not finite."""
import numpy as np
import pytest
import torch

import joint_text_image_b200 as jt
from oracle import cache as oc
from test_cache_gpu import BF16, FP16, Batch, attend, f64

pytestmark = pytest.mark.gpu


def put(bt):
    """The sequences' keys and values written to the pages once more."""
    for b, (p, n) in enumerate(bt.seqs):
        for t in range(0, p + n, bt.page):
            m, pg = min(bt.page, p + n - t), int(bt.table[b, t // bt.page])
            bt.k[pg, :m] = bt.k_seq[b][t:t + m].cuda()
            bt.v[pg, :m] = bt.v_seq[b][t:t + m].cuda()


@pytest.mark.parametrize("level", [13.0, 14.0, 14.5, 15.0, 16.0, 17.0, 20.0])
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("seqs,Hq,at", [
    ([(32767, 1)], 4, 0), ([(8000, 4)], 4, 3), ([(300, 1), (5000, 1)], 8, 100),        # up to 16 rows a kv head
    ([(5000, 40)], 4, 0), ([(32000, 20)], 4, 0), ([(2000, 150), (40, 90)], 4, 7),      # more
])
def test_one_key_far_above_all_others(seqs, Hq, at, dtype, level):
    """An attention sink: one key `level` nats above all others, which share
    one score, with a value of zero: the output is the others' small weights
    alone.  Scores are exact (one product).  Weights are rounded to the type:
    half a step of them, and in fp16, whose range is short, at least half a
    step of 2^-35 of the row's largest weight (2^-36 of |v| each); exponentials
    and sums within 4e-4.  The output is rounded once more: half a step, which
    below the type's smallest normal number (fp16: 2^-14; the outputs go down to
    1e-5) is half its smallest step, 2^-25, whatever the value."""
    bt = Batch(seqs, Hq, 1, 64, 64, dtype)
    bt.q[:, :, 0] = 8.0  # scale 1/8: a key's score is its first element
    for k, v in zip(bt.k_seq, bt.v_seq):
        k.zero_()
        k[at, :, 0] = level
        v.copy_(v.abs() + 0.5)
        v[at] = 0.0
    put(bt)
    o, lse = attend(bt)
    o, lse = f64(o), f64(lse)
    fi = torch.finfo(dtype)
    u, sub = fi.eps / 2, fi.smallest_normal * fi.eps / 2
    for b, (p, n) in enumerate(seqs):
        r, v = int(bt.rows[b]), f64(bt.v_seq[b])[:, 0]
        below = np.cumsum(v, 0)
        for i in range(n):
            s = np.zeros(p + i + 1)
            s[at if at <= p + i else 0:][:1] = level if at <= p + i else 0.0
            z = np.exp(s).sum()
            want = below[p + i] / z  # the sink's value is 0
            tol = 2 * u * 1.01 * want + 4e-4 * want + sub
            if dtype is FP16:
                tol += below[p + i] * 2.0 ** -36 * np.exp(s.max()) / z
            err = np.abs(o[r + i] - want)
            assert np.all(err <= tol), f"{(err / want).max():.2e} of the output, allowed {(tol / want).min():.2e}"
            assert np.all(np.abs(lse[:, r + i] - np.log(z)) <= 2.1e-4 + 1e-6 * abs(np.log(z)))


@pytest.mark.parametrize("seqs,Hq,Hkv", [
    ([(0, 1), (0, 3), (40, 1)], 4, 2), ([(3000, 2), (100, 4)], 8, 2),      # up to 16 rows a kv head
    ([(0, 200), (60, 90), (3, 30)], 8, 2), ([(4000, 20)], 8, 1),           # more: two row tiles, one
])
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("which", ["all", "half", "one"])
@pytest.mark.parametrize("bounded", [False, True])
def test_infinite_keys(seqs, Hq, Hkv, dtype, which, bounded):
    """Keys that hold infinities give scores of both infinities: a score of
    -inf is a weight of zero beside finite ones, a row that sees no other score
    has no weights by the formula (NaN), nor has one that sees +inf.  A row that
    sees no key at all stays empty."""
    bt = Batch(seqs, Hq, Hkv, 64, 16, dtype, seed=12)
    g = torch.Generator().manual_seed(13)
    up = torch.rand(bt.T, Hq, generator=g) < 0.3
    bt.q[:, :, 0] = torch.where(up, 1.0, -1.0).to(dtype)
    for b, (p, n) in enumerate(seqs):
        L = p + n
        bt.k_seq[b][slice(0, L) if which == "all" else slice(0, (L + 1) // 2) if which == "half" else slice(p, p + 1),
                    :, 0] = float("inf")
    put(bt)
    bound = None
    if bounded:
        bound = torch.cat([torch.randint(0, p + n, (n,), generator=g) for p, n in seqs]).int()
        bound[::7] = -1
    o, lse = attend(bt, bound)
    o, lse = f64(o), f64(lse)
    u = torch.finfo(dtype).eps / 2
    for b, (p, n) in enumerate(seqs):
        r = int(bt.rows[b])
        last = np.arange(p, p + n) if bound is None else bound[r:r + n].numpy()
        with np.errstate(invalid="ignore"):
            ro, rl, ra = oc.attend(f64(bt.q[r:r + n]), f64(bt.k_seq[b]), f64(bt.v_seq[b]), last, 0.125)
        go, gl = o[r:r + n], lse[:, r:r + n]
        assert np.array_equal(np.isnan(go), np.isnan(ro)) and np.array_equal(np.isnan(gl), np.isnan(rl))
        assert np.array_equal(np.isneginf(gl), np.isneginf(rl)) and not np.any(np.isposinf(gl))
        assert np.all(go[np.isneginf(rl).T] == 0)
        fin = np.isfinite(ro)
        assert np.all(np.abs(go[fin] - ro[fin]) <= (u * (ra + np.abs(ro)) * 1.01 + 4e-4 * ra + 1e-7)[fin])
        fin = np.isfinite(rl)
        assert np.all(np.abs(gl[fin] - rl[fin]) <= 2.1e-4 + 1e-6 * np.abs(rl[fin]))


@pytest.mark.parametrize("seqs", [[(0, 1), (300, 1), (2000, 2)], [(0, 150), (700, 90)], [(3000, 20)]])
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("q0,above", [(8192.0, True), (8192.0, False), (-8192.0, True), (-8192.0, False)])
def test_scores_of_tens_of_millions(seqs, dtype, q0, above):
    """Scores near +-6e7, one key's above all others or all equal: the one
    value, or the values' mean.  Scores are exact (one product); a row's
    largest weights are equal, each rounded to the type (half a step, as the
    output), and summed in fp32."""
    bt = Batch(seqs, 4, 1, 64, 16, dtype, seed=31)
    bt.q.zero_()
    bt.q[:, :, 0] = q0
    for b, (p, n) in enumerate(seqs):
        bt.k_seq[b].zero_()
        bt.k_seq[b][:, :, 0] = 57344.0 if above and q0 < 0 else 53248.0
        if above:
            bt.k_seq[b][p // 2, :, 0] = 53248.0 if q0 < 0 else 57344.0
    put(bt)
    o, lse = attend(bt)
    o, lse = f64(o), f64(lse)
    u = torch.finfo(dtype).eps / 2
    for b, (p, n) in enumerate(seqs):
        v = f64(bt.v_seq[b])[:, 0]
        for i in range(n):
            one = above and p // 2 <= p + i
            want = v[p // 2] if one else v[:p + i + 1].mean(0)
            a = np.abs(want) if one else np.abs(v[:p + i + 1]).mean(0)
            assert np.all(np.abs(o[int(bt.rows[b]) + i] - want) <= 1.01 * u * (a + np.abs(want)) + 4e-4 * a)
            top = q0 * (53248.0 if (q0 < 0) == bool(one) or not above else 57344.0) / 8
            assert np.all(np.abs(lse[:, int(bt.rows[b]) + i] - top) <= 1e-6 * abs(top))


@pytest.mark.parametrize("far", [1, 2])
def test_one_infinite_value_costs_little(far):
    """Chunks with a row that sees nothing, each over the same long prefix, and
    an infinite value in the last key (far == 2: in one at the prefix's start
    too): the rows that see it have it by the formula, and the call takes no
    more than a few times that of finite values (every key is looked over once
    by its tile, not once more by every row)."""
    B, n, past, Hq, D, page = 160, 20, 19968, 8, 64, 64
    g = torch.Generator(device="cuda").manual_seed(14)
    shared = past // page
    k, v = (torch.randn(shared + B, page, 1, D, generator=g, device="cuda").to(BF16) for _ in range(2))
    own = shared + torch.arange(B, device="cuda")
    table = torch.cat([torch.arange(shared, device="cuda").expand(B, -1), own[:, None]], 1).int().contiguous()
    cache = jt.hia_cache(k, v)
    chunk = jt.hia_cache_chunk(table, torch.full((B,), past, dtype=torch.int32, device="cuda"),
                               torch.arange(0, B * n + 1, n, dtype=torch.int32, device="cuda"))
    q = torch.randn(B * n, Hq, D, generator=g, device="cuda").to(BF16)
    bound = torch.arange(past, past + n, dtype=torch.int32, device="cuda").repeat(B)
    bound[3::n] = -1

    def timed():
        best = 1e9
        for _ in range(4):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            out = jt.hia_attn_cache_fwd(cache, chunk, q, bound=bound)
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b))
        return out, best

    (o0, lse0), t0 = timed()
    want = o0.clone().view(B, n, Hq, D)
    v[own, n - 1, 0, 5] = float("inf")
    want[:, n - 1, :, 5] = float("inf")
    if far == 2:
        v[0, 2, 0, 9] = -float("inf")
        want[..., 9] = -float("inf")
        want[:, 3] = 0.0
    (o1, lse1), t1 = timed()
    assert jt.hia_get_device_status() == 0
    assert torch.equal(o1.view_as(want), want) and torch.equal(lse1, lse0)
    assert t1 <= 5 * t0 + 0.5, f"{t1:.3f} ms with an infinite value, {t0:.3f} without"
