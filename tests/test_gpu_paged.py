"""GPU parity of the scaled rotary tables, the per-head norms with rotation
and the paged cache's append and read, against 64-bit forms, through the C
ABI."""

import numpy as np
import pytest

import paged_ref as ref
from fp8_transformer_block_b200.synth import bf16_bits, bf16_value

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rt():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from fp8_transformer_block_b200 import build
    build.build()
    from fp8_transformer_block_b200 import frt, runtime
    return frt, runtime, torch


def status(frt):
    return frt.frt_device_status(True)


# ------------------------------------------------------------------ table ---

@pytest.mark.parametrize("M,rot,P,theta,scaling,factor,amp", [
    (1, 2, 0, 1e4, 0, 1.0, 1.0), (64, 64, 0, 1e4, 0, 1.0, 1.0), (50, 256, 816, 1e4, 0, 1.0, 1.0),
    (33, 34, 5, 1e4, 1, 4.0, 1.0), (513, 128, 1000000, 5e5, 3, 8.0, 1.2079), (100, 6, 0, 1e4, 2, 3.5, 1.0),
    (1021, 96, 131000, 1e6, 2, 16.0, 1.0), (40000, 64, 3, 5e5, 3, 32.0, 0.75)])
def test_rope_table_scaled(rt, M, rot, P, theta, scaling, factor, amp):
    frt, runtime, torch = rt
    out = torch.full((M + 1, rot), 7.0, device="cuda")
    frt.frt_build_rope_table_scaled(M, rot, P, theta, scaling, factor, 8192.0, 1.0, 32.0, amp, out)
    got = out.cpu().numpy().astype(np.float64)
    want, ang = ref.table(M, rot, P, theta, scaling, factor, amp=amp)
    # one rounding to fp32, and the fp64 angle's own error: a handful of
    # 2^-53 from the power and the products
    tol = ref.F32 * np.abs(want) + 16 * 2.0 ** -53 * (np.repeat(ang, 2, 1) + 1) * amp + 2.0 ** -149
    assert np.all(np.abs(got[:M] - want) <= tol)
    assert np.all(got[M] == 7.0)


# ------------------------------------------------------------- norm + rope ---

def make_heads(rng, rows, heads, hd, pad=0):
    x = rng.standard_normal((rows, heads * hd + pad), dtype=np.float32)
    x[rows // 2] *= 40.0
    if rows > 2:
        x[rows // 3, :hd] = 0.0
    return bf16_bits(x)


CASES = [  # rows, hq, hkv, hd, rot, half, norm, pad
    (1, 1, 1, 16, 16, True, True, 0), (50, 8, 1, 256, 256, True, False, 0), (7, 3, 0, 128, 32, False, True, 8),
    (13, 0, 2, 64, 64, True, True, 0), (301, 14, 2, 80, 32, True, True, 16), (64, 5, 5, 96, 96, False, True, 0),
    (33, 2, 1, 184, 16, True, True, 8), (2500, 24, 24, 128, 128, False, True, 0),
    (2500, 9, 3, 64, 64, True, True, 0), (700, 33, 7, 256, 64, True, True, 0), (5, 4, 2, 40, 0, True, True, 0),
    (900, 16, 5, 128, 128, True, False, 8), (3, 2, 2, 24, 16, False, False, 0)]


def run_heads(rt, rng, rows, hq, hkv, hd, rot, half, norm, pad, n_pos=4096, in_place=False):
    frt, runtime, torch = rt
    heads = hq + 2 * hkv
    x = make_heads(rng, rows, heads, hd, pad)
    pos = rng.integers(0, n_pos, rows).astype(np.int32)
    qw = bf16_bits(1 + 0.2 * rng.standard_normal(hd, dtype=np.float32)) if norm else None
    kw = bf16_bits(1 + 0.2 * rng.standard_normal(hd, dtype=np.float32)) if norm else None
    tab = None
    if rot:
        tab = torch.empty(n_pos, rot, device="cuda")
        frt.frt_build_rope_table_scaled(n_pos, rot, 0, 1e4, 0, 1, 0, 0, 0, 1.0, tab)
    dev = runtime.bf16_dev(x)
    keep = [dev, tab, torch.from_numpy(pos).cuda(), None if qw is None else runtime.bf16_dev(qw),
            None if kw is None else runtime.bf16_dev(kw)]
    ld = x.shape[1]
    q = torch.full((rows + 1, max(1, hq) * hd + 8), 3.0, dtype=torch.bfloat16, device="cuda")
    k = torch.full((rows + 1, max(1, hkv) * hd + 16), 3.0, dtype=torch.bfloat16, device="cuda")
    if in_place:
        q, k = dev, dev[:, hq * hd:]
    d = runtime.qk_rope_desc(
        rows=rows, hq=hq, hkv=hkv, hd=hd, rot=rot, layout=int(half), eps=1e-6, qkv=dev, ld_qkv=ld, q_norm=keep[3],
        k_norm=keep[4], rope=tab, n_pos=n_pos, positions=keep[2], q_out=q, ld_q=q.stride(0), k_out=k,
        ld_k=k.stride(0))
    xv = bf16_value(x)[:, :heads * hd].reshape(rows, heads, hd)
    tv = tab.cpu().numpy() if rot else None
    wv = [None if w is None else bf16_value(w).astype(np.float64) for w in (qw, kw)]
    want = [ref.norm_rotate(xv[:, :hq], wv[0], 1e-6, tv, pos, rot, half),
            ref.norm_rotate(xv[:, hq:hq + hkv], wv[1], 1e-6, tv, pos, rot, half)]
    return d, keep, q, k, want, xv


def check_rows(runtime, t, rows, heads, hd, want):
    got = bf16_value(runtime.bf16_host(t))[:rows, :heads * hd].astype(np.float64).reshape(rows, heads, hd)
    v, size = want
    # one rounding to bf16; before it fp32: the norm's factor (4 roundings),
    # two products, the rotation's product and sum, on terms of `size`
    assert np.all(np.abs(got - v) <= ref.HALF_BF16 * np.abs(v) + 10 * ref.F32 * size)


@pytest.mark.parametrize("case", CASES)
def test_norm_rope(rt, case):
    frt, runtime, torch = rt
    rows, hq, hkv, hd, rot, half, norm, pad = case
    d, keep, q, k, want, _ = run_heads(rt, np.random.default_rng(rows + hd), *case)
    frt.frt_qk_norm_rope(d)
    torch.cuda.synchronize()
    check_rows(runtime, q, rows, hq, hd, want[0])
    check_rows(runtime, k, rows, hkv, hd, want[1])
    # nothing outside the rows and columns
    assert bool((q[rows] == 3).all()) and bool((q[:, hq * hd:] == 3).all())
    assert bool((k[rows] == 3).all()) and bool((k[:, hkv * hd:] == 3).all())
    assert status(frt) == frt.FRT_OK


def test_norm_rope_in_place_equals_out_of_place(rt):
    frt, runtime, torch = rt
    case = (777, 6, 2, 128, 128, True, True, 0)
    d, keep, q, k, _, _ = run_heads(rt, np.random.default_rng(1), *case)
    frt.frt_qk_norm_rope(d)
    d2, keep2, q2, k2, _, _ = run_heads(rt, np.random.default_rng(1), *case, in_place=True)
    v = keep2[0][:, 8 * 128:].clone()
    frt.frt_qk_norm_rope(d2)
    torch.cuda.synchronize()
    assert torch.equal(q[:777, :768], q2[:, :768]) and torch.equal(k[:777, :256], k2[:, :256])
    assert torch.equal(v, keep2[0][:, 8 * 128:])


def test_norm_of_special_rows(rt):
    """Infinite, NaN, huge and all-zero heads: as the formula has them, and
    only in their own head."""
    frt, runtime, torch = rt
    hd, heads = 64, 6
    x = np.random.default_rng(9).standard_normal((3, heads * hd), dtype=np.float32)
    bits = bf16_bits(x).reshape(3, heads, hd)
    bits[0, 0, 5] = 0x7F80            # inf: the others 0, itself NaN
    bits[0, 1, 7] = 0x7FC0            # NaN
    bits[1, 2] = 0                    # zeros: 0 / sqrt(eps)
    bits[2, 3] = 0x7F00               # 2^127 each: the mean square is past fp32
    w = runtime.bf16_dev(np.full(hd, 0x3F80, np.uint16))
    dev = runtime.bf16_dev(bits.reshape(3, -1))
    out = torch.zeros(3, heads * hd, dtype=torch.bfloat16, device="cuda")
    d = runtime.qk_rope_desc(rows=3, hq=heads, hkv=0, hd=hd, rot=0, layout=1, eps=1e-6, qkv=dev,
                             ld_qkv=heads * hd, q_norm=w, q_out=out, ld_q=heads * hd)
    frt.frt_qk_norm_rope(d)
    torch.cuda.synchronize()
    g = bf16_value(runtime.bf16_host(out)).reshape(3, heads, hd)
    assert np.isnan(g[0, 0, 5]) and np.all(np.delete(g[0, 0], 5) == 0)
    assert np.all(np.isnan(g[0, 1]))
    assert np.all(g[1, 2] == 0) and np.all(g[2, 3] == 0)
    ok = np.ones((3, heads), bool)
    ok[0, 0] = ok[0, 1] = ok[1, 2] = ok[2, 3] = False
    v, size = ref.norm_rotate(bf16_value(bits), np.ones(hd), 1e-6, None, None, 0, True)
    assert np.all((np.abs(g - v) <= ref.HALF_BF16 * np.abs(v) + 10 * ref.F32 * size)[ok])


def test_positions_outside_the_table(rt):
    frt, runtime, torch = rt
    d, keep, q, k, want, _ = run_heads(rt, np.random.default_rng(2), 9, 2, 1, 64, 64, True, False, 0, n_pos=32)
    good = keep[2].clone()
    keep[2][3], keep[2][7] = -1, 32
    frt.frt_qk_norm_rope(d)
    torch.cuda.synchronize()
    assert status(frt) == frt.FRT_ERANGE and status(frt) == frt.FRT_OK
    for r in (3, 7):
        assert bool((q[r] == 3).all()) and bool((k[r] == 3).all())
    keep[2].copy_(good)
    before = q.clone()
    frt.frt_qk_norm_rope(d)
    torch.cuda.synchronize()
    rest = [0, 1, 2, 4, 5, 6, 8]
    assert torch.equal(before[rest], q[rest])
    check_rows(runtime, q, 9, 2, 64, want[0])


# ------------------------------------------------------------------- pages ---

def page_fields(rt, fmt, rng, rows, hkv, hd, ps, scales=(0.0017391147, 0.03125), spare=2):
    frt, runtime, torch = rt
    n_pages = (rows + ps - 1) // ps + spare
    slots = rng.permutation(n_pages * ps)[:rows].astype(np.int64)
    pool = torch.full((n_pages, hkv, frt.frt_kv_record_bytes(fmt, ps, hd)), 0xA5, dtype=torch.uint8,
                      device="cuda")
    kv = [torch.full((rows, hkv * hd), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    keep = [torch.from_numpy(slots).cuda(), runtime.scale_dev(scales[0]), runtime.scale_dev(scales[1])]
    f = dict(format=fmt, page_size=ps, n_pages=n_pages, pool=pool, slots=keep[0], k_scale=keep[1],
             v_scale=keep[2])
    return f, slots, pool, kv, keep


def record_rows(pool, fmt, hkv, hd, ps, slots):
    """Bytes of the slots' rows: (k codes, k scales, v codes, v scales) or (k, v)."""
    p = pool.cpu().numpy()
    page, at = slots // ps, slots % ps
    if fmt == 0:
        b = p.view(np.uint16).reshape(p.shape[0], hkv, 2, ps, hd)
        return b[page, :, 0, at], b[page, :, 1, at]
    half = p.shape[-1] // 2
    out = []
    for part in (p[..., :half], p[..., half:]):
        out.append(part[..., :ps * hd // 2].reshape(-1, hkv, ps, hd // 2)[page, :, at])
        out.append(part[..., ps * hd // 2:].reshape(-1, hkv, ps, hd // 16)[page, :, at])
    return out


@pytest.mark.parametrize("fmt,case,ps", [
    (0, (50, 8, 1, 256, 256, True, False, 0), 16), (1, (50, 8, 1, 256, 256, True, False, 0), 16),
    (1, (1, 4, 2, 64, 64, False, True, 0), 32), (0, (13, 2, 2, 72, 64, True, True, 8), 32),
    (1, (301, 14, 2, 80, 32, True, True, 16), 128), (1, (2100, 8, 4, 128, 128, True, True, 0), 64),
    (0, (2100, 8, 4, 128, 128, False, True, 0), 1024), (1, (37, 2, 1, 16, 0, True, False, 0), 16),
    (1, (900, 3, 3, 208, 48, False, True, 0), 256)])
def test_append_and_read(rt, fmt, case, ps):
    frt, runtime, torch = rt
    rows, hq, hkv, hd, rot, half, norm, pad = case
    rng = np.random.default_rng(rows * 7 + hd)
    d, keep, q, k, want, xv = run_heads(rt, rng, *case)
    frt.frt_qk_norm_rope(d)
    torch.cuda.synchronize()
    q1, k1 = q.clone(), bf16_value(runtime.bf16_host(k))[:rows, :hkv * hd].reshape(rows, hkv, hd)
    f, slots, pool, kv, keep2 = page_fields(rt, fmt, rng, rows, hkv, hd, ps)
    skip = rng.random(rows) < 0.1     # tokens without a cache row
    slots_in = np.where(skip, -1, slots)
    keep2[0].copy_(torch.from_numpy(slots_in))
    q.fill_(3.0)
    for key, val in f.items():
        setattr(d, key, frt.ptr(val) if hasattr(val, "data_ptr") else val)
    before = pool.clone()
    frt.frt_paged_kv_append(d)
    torch.cuda.synchronize()
    assert status(frt) == frt.FRT_OK
    assert torch.equal(q, q1)
    live = ~skip
    v = xv[:, hq + hkv:]
    got = record_rows(pool, fmt, hkv, hd, ps, slots)
    if fmt == 0:
        expect = [bf16_bits(k1), bf16_bits(v)]
        values = [k1, v]
    else:
        expect, values = [], []
        for x, sc in ((k1, 0.0017391147), (v, 0.03125)):
            c, s8 = ref.quantise(x, sc)
            expect += [ref.pack_codes(c), s8.astype(np.uint8)]
            y = (ref.E2M1[c] * np.repeat(ref.E4M3[s8], 16, -1)).astype(np.float32) * np.float32(sc)
            values.append(bf16_value(bf16_bits(y)))
    for g, e in zip(got, expect):
        assert np.array_equal(g[live], e[live])
    # every other byte of the pool is as it was
    shadow = before.cpu().numpy()
    page, at = slots[live] // ps, slots[live] % ps
    if fmt == 0:
        b = shadow.view(np.uint16).reshape(shadow.shape[0], hkv, 2, ps, hd)
        b[page, :, 0, at], b[page, :, 1, at] = expect[0][live], expect[1][live]
    else:
        hb = shadow.shape[-1] // 2
        for i in range(2):
            part = shadow[..., i * hb:(i + 1) * hb]
            for j, e in enumerate(expect[2 * i:2 * i + 2]):
                w = e.shape[-1]
                lo = 0 if j == 0 else ps * hd // 2
                for h in range(hkv):
                    for col in range(w):
                        part[page, h, lo + at * w + col] = e[live][:, h, col]
    assert np.array_equal(shadow, pool.cpu().numpy())
    # and back
    d.k_out, d.ld_k, d.v_out, d.ld_v = frt.ptr(kv[0]), hkv * hd, frt.ptr(kv[1]), hkv * hd
    frt.frt_paged_kv_read(d)
    torch.cuda.synchronize()
    for t, x in zip(kv, values):
        g = bf16_value(runtime.bf16_host(t)).reshape(rows, hkv, hd)
        assert np.array_equal(g[live], x[live]) and np.all(g[skip] == 3.0)


def test_append_special_values(rt):
    """Zero, subnormal, infinite and NaN elements, exact ties, saturation."""
    frt, runtime, torch = rt
    hd, ps = 64, 16
    x = np.zeros((6, 3 * hd), np.float32)   # q, k, v heads; one token a case
    kv = x[:, hd:].reshape(6, 8, 16)
    kv[0, :, :] = np.array([6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -.75, -1.25, -1.75, -2.5, -3.5, -5, 0])
    kv[1, :, 3] = np.inf
    kv[2, :, 5] = np.nan
    kv[2, :, 6] = 12.0
    kv[3] = 2.0 ** -120                      # scale rounds to 0
    kv[4, :, 0] = 3e38                       # scale saturates
    kv[5, :, 1] = -0.0
    bits = bf16_bits(np.where(np.isfinite(x), x, 0))
    bits[~np.isfinite(x)] = np.where(np.isnan(x[~np.isfinite(x)]), 0x7FC0, 0x7F80)
    dev = runtime.bf16_dev(bits)
    f, slots, pool, out, keep = page_fields(rt, 1, np.random.default_rng(3), 6, 1, hd, ps, scales=(1.0, 1.0))
    d = runtime.qk_rope_desc(rows=6, hq=1, hkv=1, hd=hd, rot=0, layout=0, eps=1e-6, qkv=dev, ld_qkv=3 * hd,
                             k_out=out[0], ld_k=hd, v_out=out[1], ld_v=hd, **f)
    frt.frt_paged_kv_append(d)
    frt.frt_paged_kv_read(d)
    torch.cuda.synchronize()
    g = bf16_value(runtime.bf16_host(out[0])).reshape(6, 4, 16)
    assert np.array_equal(g, bf16_value(runtime.bf16_host(out[1])).reshape(6, 4, 16))
    assert np.array_equal(g[0, 0], [6, 0, 1, 1, 2, 2, 4, 4, 0, -1, -1, -2, -2, -4, -4, 0])
    assert np.all(g[1, :, 3] == 2688) and np.all(np.delete(g[1], 3, 1) == 0)
    assert np.all(np.isfinite(g[2])) and np.all(g[2, :, 6] == 12.0)
    assert np.all(g[3] == 0) and np.all(g[4, :, 0] == 2688) and np.all(g[5] == 0)


def test_slots_past_the_pool(rt):
    frt, runtime, torch = rt
    for fmt in (0, 1):
        rng = np.random.default_rng(4)
        d, keep, q, k, want, _ = run_heads(rt, rng, 5, 2, 1, 64, 64, True, False, 0)
        f, slots, pool, kv, keep2 = page_fields(rt, fmt, rng, 5, 1, 64, 16)
        for key, val in f.items():
            setattr(d, key, frt.ptr(val) if hasattr(val, "data_ptr") else val)
        keep2[0].fill_(-1)
        keep2[0][2], keep2[0][4] = f["n_pages"] * 16, 1 << 60
        before = pool.clone()
        frt.frt_paged_kv_append(d)
        torch.cuda.synchronize()
        assert status(frt) == frt.FRT_ERANGE and torch.equal(before, pool)
        check_rows(runtime, q, 5, 2, 64, want[0])   # q is written all the same
        d.k_out, d.ld_k, d.v_out = frt.ptr(kv[0]), 64, None
        frt.frt_paged_kv_read(d)
        torch.cuda.synchronize()
        assert status(frt) == frt.FRT_ERANGE and bool((kv[0] == 3).all()) and status(frt) == frt.FRT_OK


def test_pool_past_32_bits(rt):
    """Slots whose byte and element offsets pass 2^32."""
    frt, runtime, torch = rt
    hkv, hd, ps, rows = 2, 256, 1024, 40
    rec = frt.frt_kv_record_bytes(1, ps, hd)
    n_pages = (9 << 30) // (hkv * rec)
    pool = torch.empty(n_pages, hkv, rec, dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(5)
    d, keep, q, k, want, xv = run_heads(rt, rng, rows, 0, hkv, hd, 256, True, False, 0)
    slots = torch.tensor([n_pages * ps - 1 - 7 * i for i in range(rows)], device="cuda")
    s = runtime.scale_dev(0.25)
    kv = [torch.zeros(rows, hkv * hd, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    d.format, d.page_size, d.n_pages, d.pool, d.slots = 1, ps, n_pages, frt.ptr(pool), frt.ptr(slots)
    d.k_scale = d.v_scale = frt.ptr(s)
    d.k_out, d.ld_k, d.v_out, d.ld_v = frt.ptr(kv[0]), hkv * hd, frt.ptr(kv[1]), hkv * hd
    frt.frt_paged_kv_append(d)
    frt.frt_paged_kv_read(d)
    torch.cuda.synchronize()
    c, s8 = ref.quantise(xv[:, hkv:], 0.25)
    v = ref.E2M1[c] * np.repeat(ref.E4M3[s8], 16, -1) * 0.25
    assert np.array_equal(bf16_value(runtime.bf16_host(kv[1])).reshape(v.shape), v)


def test_heads_on_another_stream_and_in_a_graph(rt):
    frt, runtime, torch = rt
    case = (301, 8, 2, 128, 128, True, True, 0)
    rng = np.random.default_rng(6)
    d, keep, q, k, want, _ = run_heads(rt, rng, *case)
    f, slots, pool, kv, keep2 = page_fields(rt, 1, rng, 301, 2, 128, 64)
    for key, val in f.items():
        setattr(d, key, frt.ptr(val) if hasattr(val, "data_ptr") else val)
    d.k_out, d.ld_k, d.v_out, d.ld_v = frt.ptr(kv[0]), 256, frt.ptr(kv[1]), 256
    frt.frt_paged_kv_append(d)
    frt.frt_paged_kv_read(d)
    torch.cuda.synchronize()
    q1, p1, k1 = q.clone(), pool.clone(), kv[0].clone()
    s = torch.cuda.Stream()
    q.fill_(3.0); pool.fill_(0xA5); kv[0].fill_(0)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        frt.frt_paged_kv_append(d)
        frt.frt_paged_kv_read(d)
    s.synchronize()
    assert torch.equal(q, q1) and torch.equal(pool, p1) and torch.equal(kv[0], k1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        frt.frt_paged_kv_append(d)
        frt.frt_paged_kv_read(d)
    for _ in range(2):
        q.fill_(3.0); pool.fill_(0xA5); kv[0].fill_(0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(q, q1) and torch.equal(pool, p1) and torch.equal(kv[0], k1)
