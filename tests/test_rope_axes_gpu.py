"""GPU tests of the rotary positions with several axes against the fp64 oracle.

Tolerance.  y = l c - r s (and r c + l s) in fp32 from cos, sin of absolute
error <= 4e-7 (sincospi of 2 ulp of 1, the angle's fraction rounded to fp32
and corrected to first order, its fp64 reduction <= 1e-9 for positions up to
10^6) and three roundings of 2^-24: within 1e-6 (|l| + |r|).  Then one rounding
to the type: eps/2 of the value (the same factor on the first part is in the
margin), or half the smallest step where the value is subnormal (fp16)."""
import numpy as np
import pytest
import torch

import joint_text_image_b200 as jt
from oracle import cache as oc

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def cuda_ready():
    assert torch.cuda.is_available(), "needs a GPU"
    jt.lib()


def f64(t):
    return t.detach().double().cpu().numpy()


def close(got, x, ref, dtype):
    h = x.shape[-1] // 2
    mag = np.abs(x[..., :h]) + np.abs(x[..., h:])
    mag = np.concatenate([mag, mag], -1)
    fi = torch.finfo(dtype)
    tol = fi.eps / 2 * np.abs(ref) + 1.01e-6 * mag + fi.smallest_normal * fi.eps / 2
    assert np.all(np.abs(got - ref) <= tol), np.abs(got - ref).max()


def inputs(T, Hq, Hkv, D, axes, dtype, far, seed=0):
    g = torch.Generator().manual_seed(seed)
    pos = torch.randint(-far // 8, far, (T, axes), generator=g, dtype=torch.int32)
    q = torch.randn(T, Hq, D, generator=g).to(dtype)
    k = torch.randn(T, Hkv, D, generator=g).to(dtype)
    return pos, q, k


CASES = [  # T, Hq, Hkv, D, axes, sections, per_axis, dtype, far
    (1, 1, 1, 16, 1, None, False, BF16, 100),
    (1, 32, 8, 128, 2, None, False, BF16, 10000),
    (33, 32, 8, 128, 2, None, False, FP16, 10000),
    (7, 4, 1, 64, 3, [8, 12, 12], True, FP32, 1000000),
    (515, 5, 5, 64, 3, [8, 12, 12], False, BF16, 4096),
    (129, 6, 2, 128, 4, [1, 2, 3, 58], True, FP32, 4096),
    (65, 7, 7, 96, 2, None, False, FP16, 4096),          # a head of 6 lanes
    (64, 3, 1, 256, 3, [0, 100, 28], False, BF16, 4096),  # the widest head
    (17, 2, 1, 48, 3, None, False, FP32, 4096),
    (4001, 15, 5, 80, 2, [13, 27], True, BF16, 4096),
]


@pytest.mark.parametrize("T,Hq,Hkv,D,axes,sections,per_axis,dtype,far", CASES)
@pytest.mark.parametrize("backward", [False, True])
def test_rotation(T, Hq, Hkv, D, axes, sections, per_axis, dtype, far, backward):
    pos, q, k = inputs(T, Hq, Hkv, D, axes, dtype, far)
    plan = jt.hia_rope_plan(D, axes, sections=sections, per_axis=per_axis)
    f = jt.hia_rope_axes_bwd if backward else jt.hia_rope_axes_fwd
    qo, ko = f(plan, pos.cuda(), q.cuda(), k.cuda())
    pairs = oc.rope_pairs(D, axes, sections, 10000.0, per_axis)
    for x, y in ((q, qo), (k, ko)):
        assert y.dtype == dtype and y.shape == x.shape
        close(f64(y), f64(x), oc.rotate(f64(x), pos.numpy(), pairs, -1.0 if backward else 1.0), dtype)


def test_far_positions():
    """Positions up to the ends of int32.  The fp64 reduction of 2^31 radians
    leaves 2^31 / (2 pi) * 2^-52 turns (two fp64 roundings) = 4.8e-7 radians."""
    D, T = 64, 64
    pos = torch.tensor([[2 ** 31 - 1 - i, -2 ** 31 + i] for i in range(T)], dtype=torch.int32)
    q = torch.randn(T, 2, D, generator=torch.Generator().manual_seed(3))
    plan = jt.hia_rope_plan(D, 2)
    y = f64(jt.hia_rope_axes_fwd(plan, pos.cuda(), q.cuda()))
    ref = oc.rotate(f64(q), pos.numpy(), oc.rope_pairs(D, 2, None, 10000.0, False))
    mag = np.abs(f64(q)[..., :32]) + np.abs(f64(q)[..., 32:])
    assert np.all(np.abs(y - ref) <= 1.6e-6 * np.concatenate([mag, mag], -1))


def test_gradient_against_differences():
    """<w, R(x + h e)> - <w, R(x - h e)> over 2h, in fp64 on the oracle, is the
    backward of w along e: fp32 kernel, so within 1e-6 of the row's magnitude."""
    D, T, H = 64, 5, 3
    pos, x, _ = inputs(T, H, 1, D, 3, FP32, 500, seed=7)
    w = torch.randn(T, H, D, generator=torch.Generator().manual_seed(8))
    plan = jt.hia_rope_plan(D, 3, sections=[10, 10, 12], per_axis=True)
    dx = f64(jt.hia_rope_axes_bwd(plan, pos.cuda(), w.cuda()))
    pairs = oc.rope_pairs(D, 3, [10, 10, 12], 10000.0, True)
    loss = lambda a: (f64(w) * oc.rotate(a, pos.numpy(), pairs)).sum()
    rng = np.random.default_rng(0)
    for _ in range(40):
        e = np.zeros((T, H, D))
        e[rng.integers(T), rng.integers(H), rng.integers(D)] = 1e-3
        d = (loss(f64(x) + e) - loss(f64(x) - e)) / 2e-3
        # the map is linear: differences are exact up to fp64 cancellation (1e-9)
        assert abs(d - (dx * e).sum() / 1e-3) <= 1e-5


def test_forward_then_backward_is_the_identity():
    pos, q, k = inputs(100, 8, 2, 128, 3, FP32, 5000)
    plan = jt.hia_rope_plan(128, 3, sections=[16, 24, 24])
    y = jt.hia_rope_axes_fwd(plan, pos.cuda(), q.cuda(), k.cuda())
    z = jt.hia_rope_axes_bwd(plan, pos.cuda(), *y)
    for a, b in zip((q, k), z):
        mag = a.abs()[..., :64] + a.abs()[..., 64:]
        assert torch.all((b.cpu() - a).abs() <= 4e-6 * torch.cat([mag, mag], -1))  # two passes, each within 1e-6 x 2


def test_strides_and_untouched_neighbours():
    """Views of a fused [T, Hkv, g + 2, D] projection in and out: only the rows
    of q and k change."""
    T, Hkv, g, D = 37, 3, 4, 64
    fused = torch.randn(T, Hkv, g + 2, D, generator=torch.Generator().manual_seed(1)).to(BF16).cuda()
    out = torch.full((T, Hkv, g + 2, D), 7.0, dtype=BF16, device="cuda")
    pos = torch.randint(0, 999, (T, 2), dtype=torch.int32, device="cuda")
    plan = jt.hia_rope_plan(D, 2)
    jt.hia_rope_axes_fwd(plan, pos, fused[:, :, :g], fused[:, :, g], q_out=out[:, :, :g], k_out=out[:, :, g])
    q, k = jt.hia_rope_axes_fwd(plan, pos, fused[:, :, :g].reshape(T, Hkv * g, D), fused[:, :, g].contiguous())
    assert torch.equal(out[:, :, :g].reshape(T, Hkv * g, D), q) and torch.equal(out[:, :, g], k)
    assert torch.all(out[:, :, g + 1] == 7.0)


@pytest.mark.parametrize("T", [1, 40, 5000])
def test_in_place_and_repeatable(T):
    pos, q, k = inputs(T, 8, 2, 128, 2, BF16, 5000)
    plan = jt.hia_rope_plan(128, 2)
    pos, q, k = pos.cuda(), q.cuda(), k.cuda()
    a = jt.hia_rope_axes_fwd(plan, pos, q, k)
    q2, k2 = q.clone(), k.clone()
    jt.hia_rope_axes_fwd(plan, pos, q2, k2, q_out=q2, k_out=k2)
    assert torch.equal(a[0], q2) and torch.equal(a[1], k2)
    assert torch.equal(jt.hia_rope_axes_fwd(plan, pos, q), a[0])  # q alone


def test_no_rows():
    plan = jt.hia_rope_plan(64, 2)
    q = torch.empty(0, 4, 64, dtype=BF16, device="cuda")
    assert jt.hia_rope_axes_fwd(plan, torch.empty(0, 2, dtype=torch.int32, device="cuda"), q).shape == (0, 4, 64)


def test_tables_are_those_of_the_2d_rope():
    """Interleaved axes (x, y) of a sample with an image: bit-equal to
    hia_rope2d_tables, and the rotation by them is the attention's own."""
    samples, D = [(21, 5, 7, 4)], 128
    L = 21 + 35 + 4
    seg = jt.hia_segments_build(samples, L)
    c, s = jt.hia_rope2d_tables(seg, D)
    pos = torch.tensor([[21 + (n - 21) % 7, 21 + (n - 21) // 7] if 21 <= n < 56 else [n, n] for n in range(L)],
                       dtype=torch.int32, device="cuda")
    c2, s2 = jt.hia_rope_axes_tables(jt.hia_rope_plan(D, 2), pos)
    assert torch.equal(c[0], c2) and torch.equal(s[0], s2)


def test_training_attention_with_three_axes():
    """Tables of (time, row, column) positions into hia_attn_fwd / hia_attn_bwd:
    the same result as rotating q and k first and attending with unit tables,
    up to the rounding of the rotated rows, which both make once."""
    T, Hq, Hkv, D = 150, 4, 2, 64
    g = torch.Generator().manual_seed(5)
    q, k, v, do = (torch.randn(1, T, h, D, generator=g).to(BF16).cuda() for h in (Hq, Hkv, Hkv, Hq))
    pos = torch.stack([torch.arange(T) // 30, torch.arange(T) % 30 // 6, torch.arange(T) % 6], 1).int().cuda()
    plan = jt.hia_rope_plan(D, 3, sections=[8, 12, 12], per_axis=True)
    c, s = jt.hia_rope_axes_tables(plan, pos)
    seg = jt.hia_segments_build([(T, 0, 0, 0)], T)
    o, lse = jt.hia_attn_fwd(seg, q, k, v, c, s)
    dq, dk, dv = jt.hia_attn_bwd(seg, q, k, v, c, s, o, lse, do)
    one, zero = torch.ones_like(c), torch.zeros_like(s)
    qr, kr = jt.hia_rope_axes_fwd(plan, pos, q[0], k[0])
    o2, lse2 = jt.hia_attn_fwd(seg, qr[None], kr[None], v, one, zero)
    dqr, dkr, dv2 = jt.hia_attn_bwd(seg, qr[None], kr[None], v, one, zero, o2, lse2, do)
    dq2, dk2 = jt.hia_rope_axes_bwd(plan, pos, dqr[0], dkr[0])
    rel = lambda a, b: ((a.float() - b.float()).norm() / b.float().norm()).item()
    # rotated rows may round differently where fp32 cos/sin differ in the last
    # place (a few per ten thousand): bf16 steps on those; gradients take one
    # more rounding of 2^-8
    assert rel(o2, o) <= 2 ** -8 and rel(lse2, lse) <= 1e-4 and rel(dv2, dv) <= 2 ** -8
    assert rel(dq2[None], dq) <= 2 ** -7 and rel(dk2[None], dk) <= 2 ** -7


def test_another_stream_and_graph():
    pos, q, k = inputs(50, 8, 2, 128, 2, BF16, 5000)
    plan = jt.hia_rope_plan(128, 2)
    pos, q, k = pos.cuda(), q.cuda(), k.cuda()
    qo, ko = torch.zeros_like(q), torch.zeros_like(k)
    want = jt.hia_rope_axes_fwd(plan, pos, q, k)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        jt.hia_rope_axes_fwd(plan, pos, q, k, q_out=qo, k_out=ko)
    g.replay()
    assert torch.equal(qo, want[0]) and torch.equal(ko, want[1])
    pos += 3
    want = jt.hia_rope_axes_fwd(plan, pos, q, k)
    g.replay()
    assert torch.equal(qo, want[0]) and torch.equal(ko, want[1])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        a = jt.hia_rope_axes_fwd(plan, pos, q, k)
    torch.cuda.current_stream().wait_stream(st)
    assert torch.equal(a[0], want[0])
