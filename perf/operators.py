"""Rotary tables, per-head q/k norms with rotation, paged KV appends and
attention over a 4-bit paged cache: the cases they are timed on, their plain
forms, and their definitions in 64 bits.

The page layout, stated once: the pool is one byte tensor [n_pages, hkv,
record], a record holding one head's page_size tokens as
  bf16:  keys [page_size, hd], then values [page_size, hd];
  e2m1:  key codes [page_size, hd/2] (element 2j in the low nibble of byte
         j), key scales [page_size, hd/16] (e4m3), then the values likewise.
A slot is page * page_size + row in the page.
"""

import math

import torch

own = False

# e2m1 values by code, and both nibbles of a byte
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


# ------------------------------------------------------------------ cases ---

def listed():
    return [
        # the action expert's own cache capacity: 1024 positions, one head size
        dict(name="table_expert", op="table", M=1024, rot=256, P=0, theta=1e4, scaling="none", factor=1.0),
        # a 128k context stretched eight times, frequencies mixed by parts
        dict(name="table_long", op="table", M=131072, rot=128, P=0, theta=5e5, scaling="parts", factor=8.0),
        # the action expert's 50 tokens behind a prefix of 816, rotate-half
        dict(name="norm_rope_expert", op="norm_rope", rows=50, hq=8, hkv=1, hd=256, rot=256, half=True,
             norm=True, n_pos=1024, start=816),
        # the video block's 2 x 4096 tokens, 24 heads of 128, normed q and k
        dict(name="norm_rope_video", op="norm_rope", rows=8192, hq=24, hkv=24, hd=128, rot=128, half=False,
             norm=True, n_pos=4096, start=0),
        # an odd row count, a head size that is no power of two, 32 of its 80 rotated
        dict(name="norm_rope_partial", op="norm_rope", rows=1021, hq=14, hkv=2, hd=80, rot=32, half=True,
             norm=False, n_pos=32768, start=17),
        # the expert's tokens into a 4-bit cache
        dict(name="append_expert", op="append", rows=50, hq=8, hkv=1, hd=256, rot=256, half=True, norm=False,
             n_pos=1024, start=816, fp4=True, page_size=16),
        # one new token for each of 128 sequences, bf16 pages
        dict(name="append_decode", op="append", rows=128, hq=32, hkv=8, hd=128, rot=128, half=True, norm=True,
             n_pos=32768, start=-1, fp4=False, page_size=32),
        # a long prompt's tokens into a 4-bit cache, normed
        dict(name="append_prompt", op="append", rows=16381, hq=32, hkv=8, hd=128, rot=128, half=True, norm=True,
             n_pos=32768, start=0, fp4=True, page_size=64),
        # the expert's 50 tokens over prefix and themselves, every key visible
        dict(name="attend_expert", op="attend", seqs=1, q_min=50, q_max=50, k_min=866, k_max=866, hq=8, hkv=1,
             hd=256, page_size=16, causal=False, window=0),
        # one token each for a ragged batch over long caches
        dict(name="attend_decode", op="attend", seqs=61, q_min=1, q_max=1, k_min=700, k_max=16384, hq=32, hkv=8,
             hd=128, page_size=64, causal=True, window=0),
        # a few dozen new tokens each behind their histories, the stack's heads, a window
        dict(name="attend_chunks", op="attend", seqs=9, q_min=1, q_max=67, k_min=300, k_max=5000, hq=8, hkv=1,
             hd=64, page_size=32, causal=True, window=2048),
        # a whole prompt
        dict(name="attend_prompt", op="attend", seqs=1, q_min=8192, q_max=8192, k_min=8192, k_max=8192, hq=32,
             hkv=8, hd=128, page_size=64, causal=True, window=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["table", "norm_rope", "append", "attend", "attend"])
    if op == "table":
        scaling = rng.choice(["none", "linear", "base", "parts"])
        return dict(op=op, M=_log(rng, 600, 131072), rot=rng.choice([32, 64, 96, 128]), P=rng.choice([0, _log(rng, 1, 9000)]),
                    theta=rng.choice([1e4, 5e5, 1e6]), scaling=scaling,
                    factor=1.0 if scaling == "none" else round(rng.uniform(1.5, 16.0), 2))
    if op != "attend":
        hd = rng.choice([64, 80, 96, 128, 256])
        hkv = rng.choice([1, 2, 4, 8])
        hq = hkv * rng.choice([1, 3, 4, 8])
        rot = rng.choice([hd, 32]) if hd % 32 == 0 else 32
        start = rng.choice([-1, rng.randrange(20000)])
        # one token of each sequence (start < 0), or a prompt
        rows = _log(rng, 1, 400 if start < 0 else min(16000, 90_000_000 // ((hq + 2 * hkv) * hd)))
        c = dict(op=op, rows=rows, hq=hq, hkv=hkv, hd=hd, rot=rot, half=rng.random() < 0.5, norm=rng.random() < 0.5,
                 n_pos=32768, start=start)
        if op == "append":
            c.update(fp4=rng.random() < 0.6, page_size=rng.choice([16, 32, 64, 128]))
        return c
    hd = rng.choice([64, 128, 256])
    hkv = rng.choice([1, 2, 8])
    hq = hkv * rng.choice([1, 4, 7, 8])
    if hq * hd > 8192:
        hq = hkv
    many = rng.random() < 0.5
    k_max = _log(rng, 40, min(16000, 12000 * 128 // hd)) if many else _log(rng, 40, 5000)
    q_max = min(k_max, rng.choice([1, 1, 1, 2, 5])) if many else min(k_max, _log(rng, 2, 1500))
    causal = rng.random() < 0.7
    return dict(op=op, seqs=_log(rng, 1, 48) if many else rng.randrange(1, 3), q_min=1 if rng.random() < 0.5 else q_max,
                q_max=q_max, k_min=max(q_max, k_max // 8), k_max=k_max, hq=hq, hkv=hkv, hd=hd,
                page_size=rng.choice([16, 32, 64, 128]), causal=causal,
                window=rng.choice([0, 0, _log(rng, 50, 4000)]) if causal else 0)


# ----------------------------------------------------------------- inputs ---

def _spread(lo, hi, n, gen):
    """n whole numbers in [lo, hi], the ends among them where n allows."""
    v = torch.randint(lo, hi + 1, (n,), generator=gen)
    v[-1] = hi
    if n > 1:
        v[0] = lo
    return v


def _quantise(x, static):
    """Plain 4-bit form of x [..., hd] (fp32 values of bf16 numbers): the
    codes' and scales' bytes."""
    y = (x * (1.0 / static)).unflatten(-1, (-1, 16))
    six = torch.full((), 6.0, device=y.device)  # a tensor: by a number torch multiplies with the reciprocal
    s8 = (y.abs().amax(-1) / six).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = s8.float().unsqueeze(-1)
    t = torch.where(s > 0, y / s, torch.zeros_like(y))
    a = t.abs()
    # nearest code, a tie to the even one: the borders between neighbours
    c = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int()
         + (a >= 3.5).int() + (a > 5.0).int())
    c = (c + 8 * torch.signbit(t).int()).flatten(-2)
    return (c[..., 0::2] + 16 * c[..., 1::2]).to(torch.uint8), s8.view(torch.uint8)


def _parts(pool, hd, page_size):
    """The four parts of a 4-bit pool: key codes, key scales, value codes, value scales."""
    a, b = page_size * hd // 2, page_size * hd // 16
    k, ks, v, vs = pool.split([a, b, a, b], dim=-1)
    sh = pool.shape[:-1] + (page_size, -1)
    return k.unflatten(-1, sh[-2:]), ks.unflatten(-1, sh[-2:]), v.unflatten(-1, sh[-2:]), vs.unflatten(-1, sh[-2:])


def _table(n_pos, rot, theta=1e4):
    """A plain fp32 table [n_pos, rot], cos and sin side by side."""
    f = theta ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    a = torch.arange(n_pos, device="cuda", dtype=torch.float64)[:, None] * f
    return torch.stack([a.cos(), a.sin()], -1).flatten(-2).float()


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator("cuda").manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    s = {"case": c}

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=gen, device="cuda") * std

    if c["op"] == "table":
        # another seed is another stretch of positions
        c["P"] = c["P"] + seed % 97
        s["out"] = torch.empty(c["M"], c["rot"], device="cuda")
        return s

    hq, hkv, hd = c["hq"], c["hkv"], c["hd"]
    s["static"] = torch.tensor([0.0017391147, 0.0019013729], device="cuda")  # static key and value scales
    s["k_scale"], s["v_scale"] = s["static"][0:1], s["static"][1:2]

    if c["op"] == "attend":
        n, ps = c["seqs"], c["page_size"]
        size = torch.Generator().manual_seed(5)  # the lengths belong to the case, not to the seed
        ql, kl = _spread(c["q_min"], c["q_max"], n, size), _spread(c["k_min"], c["k_max"], n, size)
        need = (kl + ps - 1) // ps
        max_pages, n_pages = int(need.max()), int(need.sum()) + 3
        # pages in no order, those no sequence owns among them
        ids = torch.randperm(n_pages, generator=host)[:int(need.sum())].to(torch.int32)
        table = torch.zeros(n, max_pages, dtype=torch.int32)
        table[torch.arange(max_pages)[None] < need[:, None]] = ids
        cu = torch.zeros(n + 1, dtype=torch.int32)
        cu[1:] = ql.cumsum(0)
        rows = int(cu[-1])
        s["row_seq"] = torch.repeat_interleave(torch.arange(n), ql).cuda()
        s["row_i"] = (torch.arange(rows) - cu[:-1].long()[s["row_seq"].cpu()]).cuda()
        s["table"], s["cu"], s["kl"] = table.cuda(), cu.cuda(), kl.to(torch.int32).cuda()
        s["ql"], s["rows"], s["max_pages"], s["n_pages"] = ql.to(torch.int32).cuda(), rows, max_pages, n_pages
        s["q"] = normal(rows, hq, hd, std=1.3).bfloat16()
        kc, ks = _quantise(normal(n_pages, hkv, ps, hd).bfloat16().float(), s["k_scale"])
        vc, vs = _quantise(normal(n_pages, hkv, ps, hd).bfloat16().float(), s["v_scale"])
        s["pool"] = torch.cat([p.flatten(-2) for p in (kc, ks, vc, vs)], -1)
        s["out"] = torch.empty(rows, hq, hd, device="cuda", dtype=torch.bfloat16)
        s["lse"] = torch.empty(rows, hq, device="cuda")
        return s | (_handles(s) if own else {})

    rows, N = c["rows"], (hq + 2 * hkv) * hd
    s["qkv"] = normal(rows, N).bfloat16()
    s["q_norm"] = (1.0 + normal(hd, std=0.1)).bfloat16() if c["norm"] else None
    s["k_norm"] = (1.0 + normal(hd, std=0.1)).bfloat16() if c["norm"] else None
    s["rope"] = _table(c["n_pos"], c["rot"])
    if c["start"] < 0:  # a batch of sequences, each at a place of its own
        pos = torch.randint(0, c["n_pos"], (rows,), generator=host)
    else:               # consecutive tokens, wrapping like a batch of equal sequences
        pos = (c["start"] + torch.arange(rows)) % c["n_pos"]
    s["positions"] = pos.to(torch.int32).cuda()
    s["q_out"] = torch.empty(rows, hq * hd, device="cuda", dtype=torch.bfloat16)
    s["k_out"] = torch.empty(rows, hkv * hd, device="cuda", dtype=torch.bfloat16)
    if c["op"] == "append":
        ps = c["page_size"]
        n_pages = (rows + ps - 1) // ps + 2 if c["start"] >= 0 else rows + 2
        if c["start"] >= 0:    # consecutive slots through a shuffled page list
            pages = torch.randperm(n_pages, generator=host)
            slots = pages[torch.arange(rows) // ps] * ps + torch.arange(rows) % ps
        else:                  # one token in a page of each sequence
            slots = torch.randperm(n_pages, generator=host)[:rows] * ps + pos % ps
        s["slots"], s["n_pages"] = slots.cuda(), n_pages
        s["v_out"] = torch.empty_like(s["k_out"])
        if c["fp4"]:
            s["pool"] = torch.zeros(n_pages, hkv, ps * hd * 9 // 8, device="cuda", dtype=torch.uint8)
        else:
            s["pool"] = normal(n_pages, hkv, 2 * ps * hd).bfloat16().view(torch.uint8)
    return s | (_handles(s) if own else {})


# ------------------------------------------------------------ plain forms ---

def _plain_table(s):
    c = s["case"]
    rot, factor = c["rot"], c["factor"]
    theta = c["theta"] * factor ** (rot / (rot - 2)) if c["scaling"] == "base" else c["theta"]
    f = theta ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    if c["scaling"] == "linear":
        f = f / factor
    if c["scaling"] == "parts":
        keep = ((ORIG * f / (2 * math.pi) - LOW) / (HIGH - LOW)).clamp(0, 1)
        f = f * (keep + (1 - keep) / factor)
    a = torch.arange(c["P"], c["P"] + c["M"], device="cuda", dtype=torch.float64)[:, None] * f
    amp = _amplitude(c)
    return torch.stack([amp * a.cos(), amp * a.sin()], -1).flatten(-2).float()


ORIG, LOW, HIGH = 8192.0, 1.0, 32.0  # the trained context, and the turns in it that bound the ramp


def _amplitude(c):
    return 0.1 * math.log(c["factor"]) + 1.0 if c["scaling"] == "parts" else 1.0


def _norm_rotate(x, w, s):
    """Heads x [rows, heads, hd] bf16 -> normed, rotated, fp32.  The mean
    square is summed in 64 bits: a key's code may lie next to a border."""
    c, rot = s["case"], s["case"]["rot"]
    x = x.float()
    if w is not None:
        m = x.double().square().mean(-1, keepdim=True).float()
        x = x * (1.0 / torch.sqrt(m + 1e-6)) * w.float()
    cs = s["rope"][s["positions"].long()].unflatten(-1, (-1, 2)).unsqueeze(1)
    co, si = cs[..., 0], cs[..., 1]
    if c["half"]:
        x0, x1 = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([x0 * co - x1 * si, x0 * si + x1 * co], -1)
    else:
        x0, x1 = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([x0 * co - x1 * si, x0 * si + x1 * co], -1).flatten(-2)
    return torch.cat([y, x[..., rot:]], -1).bfloat16()


def _plain_norm_rope(s):
    c = s["case"]
    hq, hkv, hd = c["hq"], c["hkv"], c["hd"]
    x = s["qkv"].unflatten(-1, (-1, hd))
    q = _norm_rotate(x[:, :hq], s["q_norm"], s)
    k = _norm_rotate(x[:, hq:hq + hkv], s["k_norm"], s)
    return {"q": q.flatten(1), "k": k.flatten(1)}


def _values(codes, scales, static):
    """Codes [..., hd/2] and scales [..., hd/16] -> fp32 values [..., hd]."""
    lut = torch.tensor(E2M1, device="cuda")
    pairs = torch.stack([lut.repeat(16), lut.repeat_interleave(16)], -1)
    x = pairs[codes.int()].flatten(-2).unflatten(-1, (-1, 16))
    return (x * scales.view(torch.float8_e4m3fn).float().unsqueeze(-1)).flatten(-2) * static


def _plain_append(s):
    c = s["case"]
    hq, hkv, hd, ps = c["hq"], c["hkv"], c["hd"], c["page_size"]
    q, k = _plain_norm_rope(s).values()
    k = k.unflatten(-1, (hkv, hd))
    v = s["qkv"].unflatten(-1, (-1, hd))[:, hq + hkv:]
    page, at = s["slots"] // ps, s["slots"] % ps
    if not c["fp4"]:
        kv = s["pool"].view(torch.bfloat16).view(-1, hkv, 2, ps, hd)
        kv[page, :, 0, at] = k
        kv[page, :, 1, at] = v
        return {"q": q, "pool": s["pool"].view(torch.bfloat16)}
    kc, ks, vc, vs = _parts(s["pool"], hd, ps)
    kc[page, :, at], ks[page, :, at] = _quantise(k.float(), s["k_scale"])
    vc[page, :, at], vs[page, :, at] = _quantise(v.float(), s["v_scale"])
    k = _values(kc[page, :, at], ks[page, :, at], s["k_scale"]).bfloat16()
    v = _values(vc[page, :, at], vs[page, :, at], s["v_scale"]).bfloat16()
    return {"q": q, "k": k.flatten(1), "v": v.flatten(1)}


def _plain_attend(s):
    c = s["case"]
    hq, hkv, hd, ps, n = c["hq"], c["hkv"], c["hd"], c["page_size"], c["seqs"]
    G, max_q, cap = hq // hkv, c["q_max"], s["max_pages"] * ps
    kc, ks, vc, vs = (p[s["table"].long()].transpose(1, 2).flatten(2, 3) for p in _parts(s["pool"], hd, ps))
    k = _values(kc, ks, s["k_scale"])                       # [n, hkv, cap, hd]
    v = _values(vc, vs, s["v_scale"])
    i = torch.arange(max_q, device="cuda")
    at = (s["cu"][:-1].long()[:, None] + i).clamp(max=s["rows"] - 1)
    q = s["q"].float()[at].unflatten(2, (hkv, G)).permute(0, 2, 3, 1, 4).flatten(2, 3)   # [n, hkv, G*max_q, hd]
    x = (q @ k.transpose(-1, -2)).mul_(hd ** -0.5).unflatten(2, (G, max_q))
    j = torch.arange(cap, device="cuda")
    pos = (s["kl"] - s["ql"])[:, None] + i                  # [n, max_q]
    see = (j < s["kl"][:, None])[:, None, :].expand(n, max_q, cap)
    if c["causal"]:
        see = see & (j <= pos[..., None])
    if c["window"]:
        see = see & (j > pos[..., None] - c["window"])
    x.masked_fill_(~see[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True).clamp(min=-1e30)           # a row that sees nothing stays finite
    x.sub_(m).exp_()
    z = x.sum(-1, keepdim=True)
    o = (x.flatten(2, 3) @ v).unflatten(2, (G, max_q)) / z.clamp(min=1e-38)
    lse = (m + z.log()).squeeze(-1)
    o = o.permute(0, 3, 1, 2, 4).flatten(2, 3)[s["row_seq"], s["row_i"]]
    return {"out": o.bfloat16(), "lse": lse.permute(0, 3, 1, 2).flatten(2, 3)[s["row_seq"], s["row_i"]]}


# ------------------------------------------------------ the library's calls ---

def _handles(s):
    """What a program keeps beside its buffers: descriptors and the zero-filled workspace."""
    from fp8_transformer_block_b200 import frt, runtime as rt
    c = s["case"]
    if c["op"] == "attend":
        nbytes = frt.frt_paged_attention_workspace_size(c["seqs"], c["q_max"], c["hq"], c["hkv"], c["hd"])
        ws = rt.workspace(nbytes)
        d = rt.paged_attn_desc(
            n_seqs=c["seqs"], rows=s["rows"], max_q=c["q_max"], hq=c["hq"], hkv=c["hkv"], hd=c["hd"], page_size=c["page_size"],
            max_pages=s["max_pages"], n_pages=s["n_pages"], causal=int(c["causal"]), window=c["window"], sm_scale=c["hd"] ** -0.5,
            q=s["q"], ld_q=c["hq"] * c["hd"], pool=s["pool"], page_table=s["table"], cu_rows=s["cu"], kv_len=s["kl"],
            k_scale=s["k_scale"], v_scale=s["v_scale"], out=s["out"], ld_out=c["hq"] * c["hd"], lse=s["lse"],
            workspace=ws, workspace_bytes=nbytes)
        return {"d": d, "ws": ws}
    pages = {}
    if c["op"] == "append":
        pages = dict(format=frt.FRT_PAGE_E2M1 if c["fp4"] else frt.FRT_PAGE_BF16, page_size=c["page_size"], n_pages=s["n_pages"],
                     pool=s["pool"], slots=s["slots"], k_scale=s["k_scale"], v_scale=s["v_scale"], v_out=s["v_out"],
                     ld_v=c["hkv"] * c["hd"])
    return {"d": rt.qk_rope_desc(
        rows=c["rows"], hq=c["hq"], hkv=c["hkv"], hd=c["hd"], rot=c["rot"],
        layout=frt.FRT_ROPE_HALF if c["half"] else frt.FRT_ROPE_PAIRS, eps=1e-6, qkv=s["qkv"], ld_qkv=s["qkv"].shape[1],
        q_norm=s["q_norm"], k_norm=s["k_norm"], rope=s["rope"], n_pos=c["n_pos"], positions=s["positions"],
        q_out=s["q_out"], ld_q=c["hq"] * c["hd"], k_out=s["k_out"], ld_k=c["hkv"] * c["hd"], **pages)}


def _own_run(s):
    from fp8_transformer_block_b200 import frt
    c = s["case"]
    if c["op"] == "table":
        kind = {"none": frt.FRT_ROPE_SCALE_NONE, "linear": frt.FRT_ROPE_SCALE_LINEAR, "base": frt.FRT_ROPE_SCALE_BASE,
                "parts": frt.FRT_ROPE_SCALE_PARTS}[c["scaling"]]
        frt.frt_build_rope_table_scaled(c["M"], c["rot"], c["P"], c["theta"], kind, c["factor"], ORIG, LOW, HIGH,
                                        _amplitude(c), s["out"])
        return s["out"]
    if c["op"] == "norm_rope":
        frt.frt_qk_norm_rope(s["d"])
        return {"q": s["q_out"], "k": s["k_out"]}
    if c["op"] == "append":
        frt.frt_paged_kv_append(s["d"])
        if not c["fp4"]:
            return {"q": s["q_out"], "pool": s["pool"].view(torch.bfloat16)}
        frt.frt_paged_kv_read(s["d"])
        return {"q": s["q_out"], "k": s["k_out"], "v": s["v_out"]}
    frt.frt_paged_attention_fp4(s["d"])
    return {"out": s["out"], "lse": s["lse"]}


def run(state):
    if own:
        return _own_run(state)
    return {"table": _plain_table, "norm_rope": _plain_norm_rope, "append": _plain_append,
            "attend": _plain_attend}[state["case"]["op"]](state)


# ------------------------------------------------------------------- work ---

def _lengths(c):
    """Mean query and key counts of the batch: its two ends and uniform draws between."""
    n = c["seqs"]
    def total(lo, hi):
        return hi if n == 1 else lo + hi + (n - 2) * (lo + hi) / 2
    return total(c["q_min"], c["q_max"]), total(c["k_min"], c["k_max"])


def work(case):
    c = case
    if c["op"] == "table":
        return {"bytes": 4 * c["M"] * c["rot"], "flops": 0}
    hq, hkv, hd = c["hq"], c["hkv"], c["hd"]
    if c["op"] == "attend":
        nq, nk = _lengths(c)
        per_seq = nk / c["seqs"]
        seen = min(c["window"], per_seq) if c["window"] else per_seq
        if c["causal"]:  # a query sees the keys up to its own place
            seen = min(seen, max(1.0, per_seq - nq / c["seqs"] / 2))
        read = min(nk, c["seqs"] * (c["window"] + nq / c["seqs"])) if c["window"] else nk
        return {"bytes": read * hkv * hd * 9 / 8 + nq * hq * (hd * 4 + 4), "flops": 4 * nq * seen * hq * hd}
    rows, units = c["rows"], c["hq"] + c["hkv"]
    table = min(rows, c["n_pos"]) * c["rot"] * 4
    n = rows * units * hd
    if c["op"] == "norm_rope":
        return {"bytes": 4 * n + table + 4 * rows, "flops": 8 * n}
    cached = rows * 2 * hkv * hd
    # 4-bit pages are written, then read back for the values they stand for
    moved = cached * (2 * 9 / 16 + 2) if c["fp4"] else cached * 2
    return {"bytes": rows * (hq + 2 * hkv) * hd * 2 + rows * hq * hd * 2 + table + 12 * rows + moved, "flops": 8 * n}


# -------------------------------------------------- definitions in 64 bits ---

def _exact_heads(x, w, c, s):
    x = x.double()
    if w is not None:
        x = x / (x.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt() * w.double()
    r = c["rot"]
    rows = s["rope"][s["positions"].long()].double()
    z = torch.complex(rows[:, None, 0::2].contiguous(), rows[:, None, 1::2].contiguous())
    head = x[..., :r]
    pair = torch.complex(head[..., :r // 2].contiguous(), head[..., r // 2:].contiguous()) if c["half"] else \
        torch.view_as_complex(head.unflatten(-1, (r // 2, 2)).contiguous())
    t = torch.view_as_real(pair * z)
    y = torch.cat([t[..., 0], t[..., 1]], -1) if c["half"] else t.flatten(-2)
    return torch.cat([y, x[..., r:]], -1)


def _exact_quantised(x, static):
    """The values the 4-bit form of x (bf16 numbers in 64 bits) stands for."""
    b = (x / static.double()).unflatten(-1, (-1, 16))
    s = (b.abs().amax(-1, keepdim=True) / 6).clamp(max=448.0).to(torch.float8_e4m3fn).double()
    u = torch.where(s > 0, b / s.clamp(min=1e-30), 0.0).clamp(-6, 6)
    # spacing 1/2 below 2, 1 below 4, 2 above; torch.round takes ties to even
    step = torch.where(u.abs() < 2, 0.5, torch.where(u.abs() < 4, 1.0, 2.0))
    return (torch.round(u / step) * step * s).flatten(-2) * static.double()


def _exact_pages(pool, pages, hd, ps):
    """One sequence's keys and values [hkv, tokens, hd] in 64 bits, without the static scales."""
    rec = pool[pages].transpose(0, 1)                                     # [hkv, pages, record]
    half = rec.shape[-1] // 2
    got = []
    for part in (rec[..., :half], rec[..., half:]):
        b = part[..., :ps * hd // 2].reshape(rec.shape[0], -1, hd // 2).int()
        code = torch.stack([b & 15, b >> 4], -1).flatten(-2)
        mag = code & 7
        val = torch.where(mag < 2, mag * 0.5, (2 + (mag & 1)) * torch.pow(2.0, (mag // 2 - 2).double()))
        sc = part[..., ps * hd // 2:].contiguous().view(torch.float8_e4m3fn).double().reshape(rec.shape[0], -1, hd // 16)
        got.append(torch.where(code > 7, -val, val) * sc.repeat_interleave(16, -1))
    return got


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "table":
        r, rot = c["factor"], c["rot"]
        i = torch.arange(rot // 2, device="cuda", dtype=torch.float64)
        base = math.log(c["theta"]) + (math.log(r) * rot / (rot - 2) if c["scaling"] == "base" else 0.0)
        w = torch.exp(-base * 2 * i / rot)
        if c["scaling"] == "linear":
            w = w / r
        if c["scaling"] == "parts":
            turns = ORIG * w / (2 * math.pi)
            mix = torch.clamp((turns - LOW) / (HIGH - LOW), 0.0, 1.0)
            w = mix * w + (1 - mix) * w / r
        a = torch.outer(torch.arange(c["M"], device="cuda", dtype=torch.float64) + c["P"], w)
        out = torch.empty(c["M"], rot, device="cuda", dtype=torch.float64)
        out[:, 0::2], out[:, 1::2] = a.cos() * _amplitude(c), a.sin() * _amplitude(c)
        return out
    hq, hkv, hd = c["hq"], c["hkv"], c["hd"]
    if c["op"] == "attend":
        G, ps = hq // hkv, c["page_size"]
        out = torch.zeros(s["rows"], hq, hd, device="cuda", dtype=torch.float64)
        lse = torch.full((s["rows"], hq), -math.inf, device="cuda", dtype=torch.float64)
        cu, kl = s["cu"].tolist(), s["kl"].tolist()
        for n in range(c["seqs"]):
            lo, hi, L = cu[n], cu[n + 1], kl[n]
            k, v = _exact_pages(s["pool"], s["table"][n, :(L + ps - 1) // ps].long(), hd, ps)
            k, v = k[:, :L] * s["k_scale"].double(), v[:, :L] * s["v_scale"].double()
            place = torch.arange(L - (hi - lo), L, device="cuda")[:, None]
            key = torch.arange(L, device="cuda")[None]
            hide = torch.zeros(hi - lo, L, dtype=torch.bool, device="cuda")
            if c["causal"]:
                hide |= key > place
            if c["window"]:
                hide |= key <= place - c["window"]
            for h in range(hq):
                x = s["q"][lo:hi, h].double() @ k[h // G].T / math.sqrt(hd)
                x = x.masked_fill(hide, -math.inf)
                lse[lo:hi, h] = torch.logsumexp(x, -1)
                out[lo:hi, h] = torch.exp(x - lse[lo:hi, h, None]).nan_to_num(0.0) @ v[h // G]
        return {"out": out, "lse": lse}
    x = s["qkv"].view(c["rows"], -1, hd)
    q = _exact_heads(x[:, :hq], s["q_norm"], c, s)
    k = _exact_heads(x[:, hq:hq + hkv], s["k_norm"], c, s)
    if c["op"] == "norm_rope":
        return {"q": q.flatten(1), "k": k.flatten(1)}
    v = x[:, hq + hkv:]
    if c["fp4"]:  # what is cached is the bf16 key
        return {"q": q.flatten(1), "k": _exact_quantised(k.bfloat16().double(), s["k_scale"]).flatten(1),
                "v": _exact_quantised(v.double(), s["v_scale"]).flatten(1)}
    pool = s["pool"].view(torch.bfloat16).double().view(-1, hkv, 2, c["page_size"], hd)
    pool[s["slots"] // c["page_size"], :, 0, s["slots"] % c["page_size"]] = k
    pool[s["slots"] // c["page_size"], :, 1, s["slots"] % c["page_size"]] = v.double()
    return {"q": q.flatten(1), "pool": pool.view(s["n_pages"], hkv, -1)}
