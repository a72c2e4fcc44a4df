"""GPU tests of long lines of work: batches with more row tiles than the plan's
block has threads, and with whole items that every CTA takes before its stretch,
and of what the append writes, slot by slot."""
import pytest
import torch

import joint_text_image_b200 as jt
from test_cache_gpu import BF16, FP16, Batch, attend

pytestmark = pytest.mark.gpu


def check_all(bt, o, lse, bound=None):
    """Every row against the definition in 64 bits; the tolerance of
    test_cache_gpu.py."""
    u, g, scale = torch.finfo(bt.dtype).eps / 2, bt.Hq // bt.Hkv, bt.D ** -0.5
    q = bt.q.cuda().double()
    for b, (p, n) in enumerate(bt.seqs):
        if n == 0:
            continue
        r = int(bt.rows[b])
        last = torch.arange(p, p + n) if bound is None else bound[r:r + n].long().clamp(max=p + n - 1)
        hide = torch.arange(p + n)[None, :] > last[:, None]
        hide, none = hide.cuda(), (last < 0).cuda()
        k, v = bt.k_seq[b].cuda().double(), bt.v_seq[b].cuda().double()
        for h in range(bt.Hkv):
            heads = slice(h * g, (h + 1) * g)
            for i in range(0, n, 1024):  # rows
                j = min(i + 1024, n)
                rows, empty = slice(r + i, r + j), none[i:j]
                s = torch.einsum("ngd,ld->ngl", q[rows, heads], k[:, h]) * scale
                s.masked_fill_(hide[i:j, None], -torch.inf)
                z = torch.logsumexp(s, -1)
                w = torch.exp(s - torch.where(empty[:, None], 0.0, z)[..., None])
                ro, ra = w @ v[:, h], w @ v[:, h].abs()
                go, gl = o[rows, heads].double(), lse[heads, rows].t().double()
                assert torch.all((go - ro).abs() <= u * (ra + ro.abs()) * 1.01 + 4e-4 * ra + 1e-7), f"sequence {b}, kv head {h}"
                assert torch.equal(gl == -torch.inf, empty[:, None].expand_as(gl)) and torch.all(go[empty] == 0)
                assert torch.all((gl - z)[~empty].abs() <= 2.1e-4 + 1e-6 * z[~empty].abs())


def lengths(B, past, new, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.rand(2, B, generator=g)
    return [(int(past ** a) - 1, int(new[0] + (new[1] - new[0] + 1) * b ** 2)) for a, b in x.t().tolist()]


LINES = [  # row tiles of 2 * (128 / g) tokens, times the kv heads, against 148 SMs
    (lengths(24, 3000, (1, 300), 1), 32, 8, 64, 32, FP16),      # some 350 items: one or two rounds of whole ones
    (lengths(40, 2000, (40, 700), 2), 32, 8, 64, 16, BF16),     # some 1500 of uneven length
    ([(900, 1200), (0, 1200), (5000, 600)], 32, 8, 128, 64, BF16),
    (lengths(600, 300, (17, 40), 3), 8, 2, 64, 16, BF16),       # 600 row tiles and more, many sequences
    ([(100, 17000)], 8, 1, 64, 64, FP16),                       # 532 row tiles of one sequence
    (lengths(700, 900, (1, 1), 4), 8, 2, 64, 16, FP16),         # 700 tiles of the few-rows kernel
    (lengths(1300, 200, (0, 2), 5), 8, 8, 64, 32, BF16),         # g = 1, some sequences without new tokens
]


@pytest.mark.parametrize("case", range(len(LINES)))
@pytest.mark.parametrize("bounded", [False, True])
def test_long_lines_of_work(case, bounded):
    seqs, Hq, Hkv, D, page, dtype = LINES[case]
    bt = Batch(seqs, Hq, Hkv, D, page, dtype, seed=case)
    bound = None
    if bounded:
        g = torch.Generator().manual_seed(21)
        bound = torch.cat([torch.arange(p, p + n) for p, n in seqs])
        # a third of the rows sees further (to the end), some less, some nothing
        pick = torch.rand(bt.T, generator=g)
        bound = torch.where(pick < 0.33, 1 << 29, torch.where(pick < 0.4, bound // 2, bound)).int()
        bound[torch.rand(bt.T, generator=g) < 0.01] = -1
    o, lse = attend(bt, bound)
    check_all(bt, o, lse, bound)
    again = attend(bt, bound)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("dtype,norm,turn", [(BF16, False, True), (FP16, True, True), (BF16, True, False), (FP16, False, False)])
def test_append_writes_its_slots_and_no_other(dtype, norm, turn):
    """In place, with q_out, and keys and values alone: each call writes the
    same k and v, all of them, into pages that hold a sentinel, and nothing
    else."""
    D = 64
    bt = Batch([(30, 40), (0, 7), (15, 0), (16, 1)], 8, 2, D, 16, dtype, fill=0.0)
    q, k, v = (torch.randn(bt.T, h, D, generator=torch.Generator().manual_seed(i)).to(dtype).cuda()
               for i, h in enumerate((8, 2, 2)))
    kw = {}
    if turn:
        kw.update(plan=jt.hia_rope_plan(D, 1), pos=torch.arange(3, bt.T + 3, dtype=torch.int32, device="cuda")[:, None])
    if norm:
        kw.update(qk_norm=(torch.linspace(0.5, 1.5, D, device="cuda"), torch.linspace(1.5, 0.5, D, device="cuda"), 1e-5))
    mine = torch.zeros(bt.k.shape[:2], dtype=torch.bool)
    for b, (p, n) in enumerate(bt.seqs):
        for t in range(p, p + n):
            mine[bt.table[b, t // 16], t % 16] = True
    mine = mine.cuda()
    got = []
    for how in ("beside", "in place", "alone"):
        bt.k.fill_(777.0), bt.v.fill_(777.0)
        x = q.clone()
        r = jt.hia_cache_append(bt.cache, bt.chunk, None if how == "alone" else x, k, v,
                                q_out=x if how == "in place" else None, **kw)
        assert (r is x) if how == "in place" else (r is None) if how == "alone" else torch.equal(x, q)
        torch.cuda.synchronize()
        assert jt.hia_get_device_status() == 0
        assert torch.all(bt.k[~mine] == 777.0) and torch.all(bt.v[~mine] == 777.0)
        assert torch.all(bt.k[mine] != 777.0) and torch.all(bt.v[mine] != 777.0)
        got.append((r, bt.k[mine], bt.v[mine]))
    for b, (p, n) in enumerate(bt.seqs):
        for i in range(n):
            assert torch.equal(bt.v[int(bt.table[b, (p + i) // 16]), (p + i) % 16], v[int(bt.rows[b]) + i])
    assert torch.equal(got[0][0], got[1][0])
    for r in got[1:]:
        assert torch.equal(r[1], got[0][1]) and torch.equal(r[2], got[0][2])
