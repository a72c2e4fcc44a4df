"""The operators of the generation path over a paged key/value cache, as they are measured: rotary positions with
several axes, appending a chunk of new tokens to the cache, and attention of the chunk over the cache.

`run` computes an operator in its plain form (elementary torch operations in 32 bits, angles in 64) or, with `own`
set, through the library's entry points.  Sizes follow the repository's workloads: 32 query and 8 key/value heads of
128 (4 of 64 per kv head in the small ones), 64 x 64 images after a text prefix of about a thousand tokens, two
samples (conditional and unconditional) per denoising step."""
import math
import random

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---------------------------------------------------------------- cases
def _rope(name, **kw):
    c = {"name": name, "op": "rope", "dtype": "bf16", "D": 128, "Hq": 32, "Hkv": 8, "T": 1, "axes": 2, "sections": "",
         "per_axis": False, "backward": False, "far": 8192, "base": 10000.0}
    c.update(kw)
    return c


def _append(name, **kw):
    c = {"name": name, "op": "append", "dtype": "bf16", "D": 128, "Hq": 32, "Hkv": 8, "B": 1, "past_lo": 0,
         "past_hi": 0, "new_lo": 1, "new_hi": 1, "page": 64, "head_major": True, "norm": True, "axes": 2, "lens": 1,
         "base": 10000.0}
    c.update(kw)
    return c


def _attn(name, **kw):
    c = {"name": name, "op": "attn", "dtype": "bf16", "D": 128, "Hq": 32, "Hkv": 8, "B": 1, "past_lo": 0,
         "past_hi": 0, "new_lo": 1, "new_hi": 1, "page": 64, "head_major": True, "image": False, "blank": 0,
         "lens": 1}
    c.update(kw)
    return c


def listed():
    return [
        # a batch of 33 tokens being decoded: latency
        _rope("rope_decode_33", T=33),
        # q and k of two 1024px samples (1024 text + 64 x 64 image + 2 tokens each), x and y interleaved
        _rope("rope_image_2x5122", T=2 * 5122),
        # gradients of a video clip of 9 x 45 x 80 latent tokens: time, height, width, each with its own frequencies
        _rope("rope_video_bwd_fp16", T=9 * 45 * 80, axes=3, sections="16,24,24", per_axis=True, backward=True,
              dtype="fp16"),
        # 32-bit gradients, odd token and head counts, time / height / width sharing one ladder of frequencies
        _rope("rope_fp32_bwd", T=4099, D=64, Hq=15, Hkv=5, axes=3, sections="8,12,12", backward=True, dtype="fp32"),
        # one new token for each of 32 requests
        _append("append_decode_32", B=32, past_lo=64, past_hi=8191),
        # the image tokens of a denoising step, conditional and unconditional sample
        _append("append_image_2x4098", B=2, past_lo=1023, past_hi=1025, new_lo=4098, new_hi=4098, page=128),
        # prompts of many lengths arriving together, small pages, token-major pages
        _append("append_prompts_fp16", B=24, past_lo=0, past_hi=2000, new_lo=1, new_hi=1400, page=16, dtype="fp16",
                D=64, Hq=16, Hkv=4, axes=3, norm=False, head_major=False),
        # one token after a 1023-token prompt: latency
        _attn("attn_token_1024", past_lo=1023, past_hi=1023),
        # 48 requests of very different lengths, one token each
        _attn("attn_decode_48", B=48, past_lo=64, past_hi=32767),
        # the denoising step itself: every image token sees the prefix and the whole image
        _attn("attn_image_2x4098", B=2, past_lo=1023, past_hi=1025, new_lo=4098, new_hi=4098, page=128, image=True),
        # prompt chunks of many lengths in one batch, small pages, token-major pages
        _attn("attn_prompts_fp16", B=12, past_lo=0, past_hi=9000, new_lo=1, new_hi=900, page=16, dtype="fp16", D=64,
              Hq=16, Hkv=4, head_major=False),
        # a short question after a long conversation with many images
        _attn("attn_question_131k", past_lo=131071, past_hi=131071, new_lo=17, new_hi=17),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "attn", "attn"])
    if op == "rope":
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        D = rng.choice([64, 128])
        axes = rng.choice([1, 2, 3])
        sections = ""
        if axes > 1 and rng.random() < 0.6:
            cut = sorted(rng.sample(range(1, D // 2), axes - 1))
            sections = ",".join(str(b - a) for a, b in zip([0] + cut, cut + [D // 2]))
        Hkv = rng.choice([1, 2, 4, 5, 8])
        c = _rope("", T=_log(rng, 1, 32000 if dtype != "fp32" else 16000), D=D, Hkv=Hkv, Hq=Hkv * rng.choice([1, 3, 4]),
                  axes=axes, sections=sections, per_axis=bool(sections) and rng.random() < 0.5,
                  backward=rng.random() < 0.5, far=_log(rng, 64, 1000000), dtype=dtype)
    else:
        Hkv, g, D = rng.choice([(8, 4, 128), (8, 4, 128), (4, 4, 64), (2, 7, 128), (5, 1, 64), (1, 8, 128)])
        few = rng.random() < 0.5
        B = _log(rng, 1, 48 if few else 8)
        new_hi = rng.choice([1, 1, 2, 5]) if few else _log(rng, 20, 1800)
        past_hi = _log(rng, 1, 32000 if few and B <= 16 else 6000)
        kw = dict(B=B, past_lo=rng.choice([0, past_hi // 3]), past_hi=past_hi,
                  new_lo=rng.choice([1, max(1, new_hi // 2)]), new_hi=new_hi, page=rng.choice([16, 32, 64, 128]),
                  head_major=rng.random() < 0.5, lens=rng.randrange(1 << 30), dtype=rng.choice(["bf16", "fp16"]),
                  D=D, Hkv=Hkv, Hq=Hkv * g)
        if op == "append":
            c = _append("", axes=rng.choice([1, 2, 3]), norm=rng.random() < 0.5, **kw)
        else:
            c = _attn("", image=new_hi > 20 and rng.random() < 0.5, blank=rng.choice([0, 0, 3]), **kw)
    del c["name"]
    return c


# ---------------------------------------------------------------- inputs
def _lengths(case):
    """Tokens in the cache and new tokens of every sequence: spread evenly over the logarithm of the range."""
    r = random.Random(case["lens"])
    past = [_log(r, case["past_lo"] + 1, case["past_hi"] + 1) - 1 for _ in range(case["B"])]
    new = [_log(r, case["new_lo"], case["new_hi"]) for _ in range(case["B"])]
    return past, new


def _sections(case):
    return [int(x) for x in case["sections"].split(",")] if case.get("sections") else None


def _randn(gen, *shape, dtype):
    return torch.randn(*shape, generator=gen, device="cuda").to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed * 2 + 1)
    dt, D, Hq, Hkv = _DTYPES[case["dtype"]], case["D"], case["Hq"], case["Hkv"]
    s = {"case": case}
    if case["op"] == "rope":
        T = case["T"]
        s["pos"] = torch.randint(0, case["far"], (T, case["axes"]), generator=gen, device="cuda", dtype=torch.int32)
        s["q"] = _randn(gen, T, Hq, D, dtype=dt)
        s["k"] = _randn(gen, T, Hkv, D, dtype=dt)
        if own:
            import joint_text_image_b200 as jt
            s["plan"] = jt.hia_rope_plan(D, case["axes"], sections=_sections(case), base=case["base"],
                                         per_axis=case["per_axis"])
        return s
    past, new = _lengths(case)
    B, page = case["B"], case["page"]
    T = sum(new)
    need = [(p + n + page - 1) // page for p, n in zip(past, new)]
    max_pages = max(need) + 2
    n_pages = sum(need) + 5
    order = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32).cpu()
    table = torch.full((B, max_pages), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    s["table"] = table.cuda()
    s["past"] = torch.tensor(past, dtype=torch.int32, device="cuda")
    s["rows"] = torch.tensor([sum(new[:b]) for b in range(B + 1)], dtype=torch.int32, device="cuda")
    s["span"] = (max(new), max(p + n for p, n in zip(past, new)))
    # the pool holds other requests' keys and values too; head-major or token-major pages
    shape = (n_pages, Hkv, page, D) if case["head_major"] else (n_pages, page, Hkv, D)
    s["k_pages"], s["v_pages"] = _randn(gen, *shape, dtype=dt), _randn(gen, *shape, dtype=dt)
    if case["head_major"]:
        s["k_pages"], s["v_pages"] = s["k_pages"].transpose(1, 2), s["v_pages"].transpose(1, 2)
    # q, k and v of the new tokens: slices of one fused projection [T, Hkv, g + 2, D]
    qkv = _randn(gen, T, Hkv, Hq // Hkv + 2, D, dtype=dt)
    s["q"], s["k"], s["v"] = qkv[:, :, :-2], qkv[:, :, -2], qkv[:, :, -1]
    if case["op"] == "append":
        s["pos"] = torch.randint(0, 8192, (T, case["axes"]), generator=gen, device="cuda", dtype=torch.int32)
        if case["norm"]:
            s["wq"] = 1 + 0.1 * torch.randn(D, generator=gen, device="cuda")
            s["wk"] = 1 + 0.1 * torch.randn(D, generator=gen, device="cuda")
    else:
        s["q"] = s["q"].reshape(T, Hq, D).contiguous()  # what the append step hands over
        s["bound"] = None
        if case["image"] or case["blank"]:
            # last visible cache position of every row: text rows end at themselves, an image span (from a
            # quarter of the chunk to its last but two rows) at its own end; blank rows (padding) see nothing
            bounds = []
            for p, n in zip(past, new):
                i0, i1 = (n // 4 if n < 4000 else 0, max(n - 2, 0)) if case["image"] else (0, 0)
                bounds += [-1 if i >= max(n - case["blank"], 1) else (p + i1 - 1 if i0 <= i < i1 else p + i)
                           for i in range(n)]
            s["bound"] = torch.tensor(bounds, dtype=torch.int32, device="cuda")
    if own:
        import joint_text_image_b200 as jt
        s["cache"] = jt.hia_cache(s["k_pages"], s["v_pages"])
        s["chunk"] = jt.hia_cache_chunk(s["table"], s["past"], s["rows"])
        if case["op"] == "append":
            s["plan"] = jt.hia_rope_plan(D, case["axes"], base=case["base"])
    return s


# ---------------------------------------------------------------- one pass
def _frequencies(D, axes, sections, per_axis, base, device):
    """Axis and angle per unit of position of every pair j < D / 2, in 64 bits."""
    j = torch.arange(D // 2, device=device)
    axis = j % axes if sections is None else torch.repeat_interleave(
        torch.arange(axes, device=device), torch.tensor(sections, device=device), output_size=D // 2)
    e = 2.0 * j.double() / D
    if per_axis:
        n = torch.tensor(sections, device=device)
        e = (j - (torch.cumsum(n, 0) - n)[axis]).double() / n[axis].double()
    return axis, torch.pow(torch.tensor(base, dtype=torch.float64, device=device), -e)


def _rotate(x, cos, sin, sign):
    lo, hi = x.float().chunk(2, dim=-1)
    return torch.cat([lo * cos - sign * hi * sin, hi * cos + sign * lo * sin], dim=-1)


def _angles(case, pos):
    axis, freq = _frequencies(case["D"], case["axes"], _sections(case), case.get("per_axis", False), case["base"],
                              pos.device)
    a = pos.double()[:, axis] * freq
    return a.cos().float()[:, None, :], a.sin().float()[:, None, :]


def _norm(x, w, eps):
    return w * (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps))


def _plain_rope(s):
    case = s["case"]
    cos, sin = _angles(case, s["pos"])
    sign = -1.0 if case["backward"] else 1.0
    return {"q": _rotate(s["q"], cos, sin, sign).to(s["q"].dtype), "k": _rotate(s["k"], cos, sin, sign).to(s["k"].dtype)}


def _places(s, T):
    """Sequence of every new row and its index in the chunk."""
    row = torch.arange(T, device=s["rows"].device)
    seq = torch.bucketize(row, s["rows"][1:].long(), right=True)
    return seq, row - s["rows"].long()[seq]


def _plain_append(s):
    case = s["case"]
    T, dt = s["q"].shape[0], s["q"].dtype
    cos, sin = _angles(case, s["pos"])
    q = _rotate(s["q"].reshape(T, case["Hq"], case["D"]), cos, sin, 1.0)
    k = _rotate(s["k"], cos, sin, 1.0)
    if case["norm"]:
        q, k = _norm(q, s["wq"], 1e-5), _norm(k, s["wk"], 1e-5)
    seq, i = _places(s, T)
    at = s["past"].long()[seq] + i
    page, slot = s["table"].long()[seq, at // case["page"]], at % case["page"]
    s["k_pages"][page, slot] = k.to(dt)
    s["v_pages"][page, slot] = s["v"]
    return {"q": q.to(dt), "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _plain_attn(s):
    case = s["case"]
    T, Hq, D = s["q"].shape
    B, Hkv, page = case["B"], case["Hkv"], case["page"]
    n_max, l_max = s["span"]
    pages = (l_max + page - 1) // page
    table = s["table"][:, :pages].long().clamp(min=0)
    col = torch.arange(pages * page, device=table.device)
    new = s["rows"][1:].long() - s["rows"][:-1].long()
    end = s["past"].long() + new
    held = (col < end[:, None])[:, :, None, None]
    k = torch.where(held, s["k_pages"][table].reshape(B, pages * page, Hkv, D), 0).float()
    v = torch.where(held, s["v_pages"][table].reshape(B, pages * page, Hkv, D), 0).float()
    seq, i = _places(s, T)
    q = torch.zeros(B, n_max, Hq, D, device=k.device)
    q[seq, i] = s["q"].float()
    last = torch.full((B, n_max), -1, dtype=torch.long, device=k.device)
    last[seq, i] = s["past"].long()[seq] + i if s["bound"] is None else s["bound"].long()
    last = torch.minimum(last, end[:, None] - 1)
    q = q.reshape(B, n_max, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4)
    sc = torch.matmul(q, k.permute(0, 2, 3, 1)[:, :, None]) * D ** -0.5      # [B, Hkv, g, n, l]
    sc.masked_fill_((col > last[:, :, None])[:, None, None], -math.inf)
    m = sc.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp_(sc.sub_(m))
    z = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v.permute(0, 2, 1, 3)[:, :, None]) / torch.where(z == 0, 1.0, z)
    lse = (m + torch.log(z))[..., 0]
    o = o.permute(0, 3, 1, 2, 4).reshape(B, n_max, Hq, D)[seq, i].to(s["q"].dtype)
    lse = lse.permute(0, 3, 1, 2).reshape(B, n_max, Hq)[seq, i].t().contiguous()
    return {"o": o, "lse": lse}


def _own(s):
    import joint_text_image_b200 as jt
    case = s["case"]
    if case["op"] == "rope":
        f = jt.hia_rope_axes_bwd if case["backward"] else jt.hia_rope_axes_fwd
        q, k = f(s["plan"], s["pos"], s["q"], s["k"])
        return {"q": q, "k": k}
    if case["op"] == "append":
        norm = (s["wq"], s["wk"], 1e-5) if case["norm"] else None
        q = jt.hia_cache_append(s["cache"], s["chunk"], s["q"], s["k"], s["v"], plan=s["plan"], pos=s["pos"],
                                qk_norm=norm)
        return {"q": q, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    o, lse = jt.hia_attn_cache_fwd(s["cache"], s["chunk"], s["q"], bound=s["bound"])
    return {"o": o, "lse": lse}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    return _plain_rope(state) if op == "rope" else _plain_append(state) if op == "append" else _plain_attn(state)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    D, Hq, Hkv = case["D"], case["Hq"], case["Hkv"]
    size = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "rope":
        n = case["T"] * (Hq + Hkv) * D
        return {"bytes": 2 * n * size + case["T"] * case["axes"] * 4, "flops": 3 * n}
    past, new = _lengths(case)
    T = sum(new)
    if case["op"] == "append":
        n = T * (Hq + 2 * Hkv) * D
        return {"bytes": 2 * n * size + T * case["axes"] * 4, "flops": (7 if case["norm"] else 3) * T * (Hq + Hkv) * D}
    pairs, keys = 0, 0
    for p, n in zip(past, new):
        i0, i1 = (n // 4 if n < 4000 else 0, max(n - 2, 0)) if case["image"] else (0, 0)
        seen = [min(p + n, p + i1 if i0 <= i < i1 else p + i + 1) for i in range(max(n - case["blank"], 1))]
        pairs += sum(seen)
        keys += max(seen, default=0)
    return {"bytes": 2 * keys * Hkv * D * size + 2 * T * Hq * D * size + 4 * T * Hq, "flops": 4 * D * Hq * pairs}


# ---------------------------------------------------------------- the definition, in 64 bits
def _exact_turn(case, pos, x, transpose):
    """x [T, H, D] rotated pair by pair: (x_j, x_{j + D/2}) turned by the angle of pair j."""
    D, axes = case["D"], case["axes"]
    sec = _sections(case)
    y = torch.empty_like(x)
    for j in range(D // 2):
        if sec is None:
            a, e = j % axes, 2.0 * j / D
        else:
            a, first = 0, 0
            while j >= first + sec[a]:
                first, a = first + sec[a], a + 1
            e = (j - first) / sec[a] if case.get("per_axis") else 2.0 * j / D
        t = pos[:, a].double() * case["base"] ** -e
        c, s = t.cos()[:, None], t.sin()[:, None]
        if transpose:
            s = -s
        u, w = x[:, :, j], x[:, :, j + D // 2]
        y[:, :, j] = u * c - w * s
        y[:, :, j + D // 2] = u * s + w * c
    return y


def exact(case, seed):
    s = prepare(case, seed)
    D, Hq, Hkv = case["D"], case["Hq"], case["Hkv"]
    if case["op"] == "rope":
        return {x: _exact_turn(case, s["pos"], s[x].double(), case["backward"]) for x in ("q", "k")}
    past, new = _lengths(case)
    T, page = sum(new), case["page"]
    table = s["table"].cpu().tolist()
    if case["op"] == "append":
        q = _exact_turn(case, s["pos"], s["q"].reshape(T, Hq, D).double(), False)
        k = _exact_turn(case, s["pos"], s["k"].double(), False)
        if case["norm"]:
            q = s["wq"].double() * q / torch.sqrt((q * q).sum(-1, keepdim=True) / D + 1e-5)
            k = s["wk"].double() * k / torch.sqrt((k * k).sum(-1, keepdim=True) / D + 1e-5)
        kp, vp = s["k_pages"].double(), s["v_pages"].double()
        r = 0
        for b, (p, n) in enumerate(zip(past, new)):
            at = p
            while at < p + n:  # one page at a time
                stop = min(p + n, (at // page + 1) * page)
                lo = at % page
                kp[table[b][at // page], lo:lo + stop - at] = k[r:r + stop - at]
                vp[table[b][at // page], lo:lo + stop - at] = s["v"][r:r + stop - at].double()
                r, at = r + stop - at, stop
        return {"q": q, "k_pages": kp, "v_pages": vp}
    o = torch.zeros(T, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((Hq, T), -math.inf, dtype=torch.float64, device="cuda")
    bound = None if s["bound"] is None else s["bound"].cpu().tolist()
    r = 0
    for b, (p, n) in enumerate(zip(past, new)):
        pages = table[b][:(p + n + page - 1) // page]
        k = s["k_pages"][pages].reshape(-1, Hkv, D)[:p + n].double()
        v = s["v_pages"][pages].reshape(-1, Hkv, D)[:p + n].double()
        seen = torch.tensor([p + i if bound is None else bound[r + i] for i in range(n)], device="cuda")
        hide = torch.arange(p + n, device="cuda")[None, :] > seen[:, None]
        some = seen >= 0
        for h in range(Hq):
            x = (s["q"][r:r + n, h].double() @ k[:, h // (Hq // Hkv)].T) / math.sqrt(D)
            x[hide] = -math.inf
            z = torch.logsumexp(x, dim=1)
            w = torch.exp(x - torch.where(some, z, 0.0)[:, None])
            o[r:r + n, h] = w @ v[:, h // (Hq // Hkv)]
            lse[h, r:r + n] = z
        r += n
    return {"o": o, "lse": lse}
