"""GPU parity of the paged operators where they can go wrong: blocks without
a key tile, score factors at the ends of fp32, variants chosen by the table's
size, and bytes that no other test looks at."""

import numpy as np
import pytest

import paged_ref as ref
from fp8_transformer_block_b200.synth import bf16_bits, bf16_value
from test_gpu_paged import check_rows, page_fields, record_rows, run_heads
from test_gpu_paged_attention import Problem, rt  # noqa: F401  (rt: the fixture)

pytestmark = pytest.mark.gpu


def repeat(p, times):
    """The same bits from call to call."""
    out, lse = p.out.clone(), p.lse.clone()
    torch = p.rt[2]
    for _ in range(times):
        p.out.fill_(5.0)
        p.lse.fill_(5.0)
        p.run()
        assert torch.equal(out, p.out) and torch.equal(lse, p.lse)


@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("hq,hkv,lens,causal", [
    # keys in no split of any block, with the keys split (few units) ...
    (8, 2, [(300, 0), (257, 3), (1, 5)], True), (8, 2, [(300, 0), (300, 0)], False),
    # ... and with the units filling the SMs
    (32, 8, [(300, 0), (300, 2), (64, 900)], True), (32, 8, [(300, 0), (300, 0), (40, 7)], False),
    # more splits than a short sequence has key tiles
    (8, 2, [(64, 1500), (64, 100), (64, 130), (33, 1)], False),
    (8, 2, [(64, 1500), (64, 100), (64, 130), (64, 9)], True)])
def test_blocks_without_a_key_tile(rt, hd, hq, hkv, lens, causal):  # noqa: F811
    """Hundreds of live rows in a block that has no key to read."""
    p = Problem(rt, np.random.default_rng(31), lens, hq, hkv, hd, 32, causal)
    p.run()
    p.check()
    repeat(p, 10)


@pytest.mark.parametrize("Lq", [1, 3, 60])
@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("gain,scale", [(2.0 ** -80, 0.0), (2.0 ** -126, 0.0), (2.0 ** 100, 0.0), (2.0 ** 120, 0.0),
                                        (2.0 ** -100, 1e-30), (2.0 ** -110, -1e-37), (1.0, 1e-45)])
def test_factors_below_fp32(rt, Lq, hd, gain, scale):  # noqa: F811
    """Scale times |q| from nothing to below the least fp32 number, under a
    mask: every visible key weighs the same."""
    p = Problem(rt, np.random.default_rng(32), [(Lq, 150), (1, 70), (Lq, 1)], 4, 2, hd, 16, scale=scale, q_gain=gain)
    p.run()
    p.check()


def check_far(p):
    """Where a row's largest score leads the next by more than the error of a
    score, the row's result is that key's value; weights are rounded to fp16
    once (2^-11), sums and the exponential add a few 2^-22."""
    o, lse = p.results()
    for s, (Lq, L) in enumerate(p.lens):
        k, v = p.kv[s]
        G = p.hq // p.hkv
        q = bf16_value(p.q)[p.cu[s]:p.cu[s + 1], :p.hq * p.hd].astype(np.float64).reshape(Lq, p.hq, p.hd)
        led = 0
        for i in range(Lq):
            for h in range(p.hq):
                seen = L - Lq + i + 1
                x = q[i, h] @ k[h // G][:seen].T * p.scale
                size = (np.abs(q[i, h]) @ np.abs(k[h // G][:seen]).T * abs(p.scale)).max()
                # hd products summed in fp32 (2^-23 a step, the tensor core
                # truncates), the scaling, q's fp16 form (2^-25 of its largest)
                err = (p.hd + 6) * 2.0 ** -23 * size + 2.0 ** -25 * np.abs(q[i, h]).max() * abs(p.scale) * \
                    np.abs(k[h // G]).sum(1).max()
                top = np.argsort(x)[::-1][:2]
                assert abs(lse[p.cu[s] + i, h] - x[top[0]]) <= 2 * err + np.log(seen) + 2.0 ** -22 * abs(x[top[0]])
                if seen == 1 or x[top[0]] - x[top[1]] > 2 * err + 64:
                    led += 1
                    want = v[h // G][top[0]]
                    got = o[p.cu[s] + i, h * p.hd:(h + 1) * p.hd]
                    assert np.all(np.abs(got - want) <= np.abs(want) * (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -18)), (s, i, h)
        assert led * 2 > Lq * p.hq


@pytest.mark.parametrize("Lq", [1, 60])
@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("scale", [1e6, 1e8, -1e9, 1e13, -1e20, 1e27])
def test_far_scores(rt, Lq, hd, scale):  # noqa: F811
    """Scores whose rounding is many steps of the exponent: one key a row."""
    p = Problem(rt, np.random.default_rng(33), [(Lq, 150), (1, 1), (Lq, Lq)], 4, 2, hd, 16, scale=scale)
    p.run()
    p.check()
    check_far(p)


@pytest.mark.parametrize("Lq", [1, 60])
@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("scale", [1e30, -1e33, 1e35])
def test_scores_of_fp32s_size(rt, Lq, hd, scale):  # noqa: F811
    """A row whose every score lies far below zero still sees its keys."""
    p = Problem(rt, np.random.default_rng(33), [(Lq, 150), (1, 1), (Lq, Lq)], 4, 2, hd, 16, scale=scale)
    p.run()
    p.check()
    check_far(p)


@pytest.mark.parametrize("hd,Lq", [(64, 1), (128, 1), (256, 1), (64, 3), (128, 3), (64, 60), (128, 60), (256, 60)])
def test_rows_of_different_sizes(rt, hd, Lq):  # noqa: F811
    """Rows of ordinary scores beside rows of far ones in the same tile."""
    frt, runtime, torch = rt
    p = Problem(rt, np.random.default_rng(37), [(Lq, 200), (Lq, 70)], 8, 2, hd, 16)
    p.run()
    want, lse = p.out.clone(), p.lse.clone()
    rows = np.zeros(p.q.shape, bool)
    for h in (1, 6):   # one head of each kv head, in every third row
        rows[::3, h * hd:(h + 1) * hd] = True
    p.q[rows] = bf16_bits(bf16_value(p.q)[rows] * np.float32(2.0 ** 90))
    p.t["q"].copy_(runtime.bf16_dev(p.q))
    p.run()
    p.check()
    keep = torch.from_numpy(~rows).cuda()[:, :8 * hd]
    assert torch.equal(p.out[keep], want[keep])
    assert torch.equal(p.lse[keep[:, ::hd]], lse[keep[:, ::hd]])


@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("lens,hq,hkv", [
    ([(1, 300)], 8, 2), ([(1, 9000)], 8, 2),     # few rows: a whole unit, a cut one
    ([(50, 866)], 8, 1), ([(64, 300)] * 10, 32, 8)])  # many: split keys, whole
def test_nan_in_q(rt, hd, lens, hq, hkv):  # noqa: F811
    """A NaN stays in its row and head, in out and lse alike."""
    torch = rt[2]
    p = Problem(rt, np.random.default_rng(34), lens, hq, hkv, hd, 32)
    p.run()
    out, lse = p.out.clone(), p.lse.clone()
    row, h = int(p.cu[-1]) - 1, hq - 1
    at = slice(h * hd, (h + 1) * hd)
    p.t["q"][row, h * hd + 5] = float("nan")
    p.run()
    assert bool(torch.isnan(p.out[row, at]).all()) and bool(torch.isnan(p.lse[row, h]))
    p.out[row, at], p.lse[row, h] = out[row, at], lse[row, h]
    assert torch.equal(p.out, out) and torch.equal(p.lse, lse)


@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("Lq", [1, 3, 60])
@pytest.mark.parametrize("size,scale", [(2.0 ** 127, 2.0 ** -123), (2.0 ** -131, 3e38)])
def test_q_at_the_ends_of_bf16(rt, hd, Lq, size, scale):  # noqa: F811
    """Rows whose largest |q| is 2^127 and above, and subnormal rows."""
    runtime = rt[1]
    rng = np.random.default_rng(38)
    p = Problem(rt, rng, [(Lq, 150), (1, 40)], 4, 2, hd, 16, scale=scale)
    p.q = bf16_bits(rng.uniform(-1.9, 1.9, p.q.shape).astype(np.float32) * np.float32(size))
    p.t["q"].copy_(runtime.bf16_dev(p.q))
    p.run()
    p.check()


@pytest.mark.parametrize("hd,hkv", [(64, 2), (208, 1), (256, 5)])
def test_codes_of_zeros(rt, hd, hkv):  # noqa: F811
    """The bytes of zeros of either sign, among others and alone, and of what
    rounds to zero."""
    frt, runtime, torch = rt
    rng = np.random.default_rng(35)
    rows, ps = 40, 16
    x = rng.standard_normal((rows, 2 * hkv * hd), dtype=np.float32)
    x[rng.random(x.shape) < 0.3] = -0.0
    x[rng.random(x.shape) < 0.2] = 0.0
    x[rng.random(x.shape) < 0.1] *= np.float32(2.0 ** -40)
    x[3], x[4] = -0.0, np.where(rng.random(x.shape[1]) < 0.5, 0.0, -0.0)
    bits = bf16_bits(x)
    dev = runtime.bf16_dev(bits)
    f, slots, pool, kv, keep = page_fields(rt, 1, rng, rows, hkv, hd, ps)
    frt.frt_paged_kv_append(runtime.qk_rope_desc(
        rows=rows, hq=0, hkv=hkv, hd=hd, rot=0, layout=0, eps=1e-6, qkv=dev, ld_qkv=x.shape[1], **f))
    torch.cuda.synchronize()
    got = record_rows(pool, 1, hkv, hd, ps, slots)
    v = bf16_value(bits).reshape(rows, 2, hkv, hd)
    for i, scale in enumerate((0.0017391147, 0.03125)):
        codes, s8 = ref.quantise(v[:, i], scale)
        assert np.array_equal(got[2 * i], ref.pack_codes(codes))
        assert np.array_equal(got[2 * i + 1], s8.astype(np.uint8))


def counters_are_zero(p):
    """All of the workspace's head that a later call could find counters in."""
    head = p.ws[:4096].view(p.rt[2].int32)
    assert head.numel() == 1024 and int(head.abs().sum()) == 0


@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("hq,hkv,Lq", [(8, 1, 1), (8, 2, 2), (16, 1, 1), (12, 1, 1), (8, 2, 4), (3, 1, 5), (32, 1, 1),
                                       (4, 2, 15), (8, 1, 3)])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 130)])
def test_table_capacities(rt, hd, hq, hkv, Lq, causal, window):  # noqa: F811
    """1 to 32 rows of a kv head over a table just wide enough and over a wide
    one: 9 to 32 rows go to one kernel or the other by the table's width."""
    for extra in (0, 80):
        p = Problem(rt, np.random.default_rng(36), [(Lq, 1300), (Lq, 64), (1, 513), (Lq, Lq), (0, 90)], hq, hkv, hd, 64,
                    causal, window, extra_pages=extra)
        p.run()
        p.check()
        counters_are_zero(p)


@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("hq,hkv", [(8, 1), (16, 1), (24, 1), (8, 8)])
@pytest.mark.parametrize("lens", [[(1, 20000)], [(1, 5000), (1, 1), (1, 3333)] * 9])
def test_cut_units_leave_counters_at_zero(rt, hd, hq, hkv, lens):  # noqa: F811
    p = Problem(rt, np.random.default_rng(39), lens, hq, hkv, hd, 128)
    p.run()
    p.check()
    counters_are_zero(p)
    repeat(p, 3)
    counters_are_zero(p)


@pytest.mark.parametrize("Lq", [1, 5, 200])
def test_rows_of_bad_row_offsets(rt, Lq):  # noqa: F811
    """Row offsets that run backwards, past the tensor or past max_q: the
    rows that are left of each sequence, and nothing else, are written."""
    frt, runtime, torch = rt
    p = Problem(rt, np.random.default_rng(40), [(Lq, 600), (Lq, 300)], 4, 1, 64, 64, causal=False)
    q = bf16_value(p.q).astype(np.float64).reshape(p.rows, 4, 64)
    for cu in ([0, Lq, 5 * Lq + 99], [-4, Lq, 2 * Lq], [0, Lq, 0], [2 ** 30, Lq, 2 * Lq], [0, 2 ** 31 - 1, 2 ** 31 - 1],
               [-2 ** 31, -1, 2 * Lq], [Lq, 0, Lq], [p.rows, p.rows + 1, 0]):
        p.t["cu_rows"].copy_(torch.tensor(cu, dtype=torch.int32))
        p.out.fill_(5.0)
        p.lse.fill_(5.0)
        p.run(report=False)
        assert frt.frt_device_status(True) == frt.FRT_ERANGE
        o, lse = p.results()
        left = np.ones(p.rows, bool)
        for s in range(2):
            lo = min(max(cu[s], 0), p.rows)
            hi = min(max(cu[s + 1], lo), p.rows, lo + Lq)
            if hi == lo:
                continue
            # no two of these ranges overlap
            assert np.all(left[lo:hi])
            left[lo:hi] = False
            k, v = p.kv[s]
            want, wl, tol, tl = ref.attention(q[lo:hi], k, v, p.lens[s][1], False, 0, p.scale)
            got = o[lo:hi].reshape(want.shape)
            assert np.all(np.abs(got - want) <= ref.HALF_BF16 * np.abs(want) + tol), (cu, s)
            assert np.all(np.abs(lse[lo:hi] - wl) <= tl)
        assert np.all(o[left] == 5.0) and np.all(lse[left] == 5.0), cu


@pytest.mark.parametrize("ps", [16, 64, 1024])
@pytest.mark.parametrize("lens", [[(1, 700), (1, 130)], [(5, 700), (2, 70)], [(70, 700), (3, 90)]])
def test_attention_over_a_pool_past_32_bits(rt, lens, ps):  # noqa: F811
    """Pages whose byte offsets pass 2^32, in every kernel's copies."""
    frt, runtime, torch = rt
    p = Problem(rt, np.random.default_rng(41), lens, 8, 2, 256, ps)
    small = p.t["pool"]
    n_pages = (5 << 30) // small[0].numel()
    pool = torch.empty(n_pages, *small.shape[1:], dtype=torch.uint8, device="cuda")
    pool[n_pages - p.n_pages:] = small.flip(0)
    table = torch.from_numpy(np.where(p.table >= 0, n_pages - 1 - p.table, p.table))
    p.t["page_table"].copy_(table)
    p.d.pool, p.d.n_pages = frt.ptr(pool), n_pages
    p.run()
    p.check()


def test_keys_past_32_bits(rt):  # noqa: F811
    """Appended and read back where slots' byte offsets pass 2^32, keys and
    values alike, in both formats."""
    frt, runtime, torch = rt
    hkv, hd, ps, rows = 2, 256, 1024, 40
    rng = np.random.default_rng(42)
    x = bf16_bits(rng.standard_normal((rows, 2 * hkv * hd), dtype=np.float32))
    dev = runtime.bf16_dev(x)
    v = bf16_value(x).reshape(rows, 2, hkv, hd)
    scale = runtime.scale_dev(0.25)
    for fmt in (0, 1):
        rec = frt.frt_kv_record_bytes(fmt, ps, hd)
        n_pages = (9 << 30) // (hkv * rec)
        pool = torch.empty(n_pages, hkv, rec, dtype=torch.uint8, device="cuda")
        slots = torch.tensor([n_pages * ps - 1 - 7 * i for i in range(rows)], device="cuda")
        kv = [torch.zeros(rows, hkv * hd, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        d = runtime.qk_rope_desc(
            rows=rows, hq=0, hkv=hkv, hd=hd, rot=0, layout=0, eps=1e-6, qkv=dev, ld_qkv=x.shape[1], format=fmt,
            page_size=ps, n_pages=n_pages, pool=pool, slots=slots, k_scale=scale, v_scale=scale, k_out=kv[0],
            ld_k=hkv * hd, v_out=kv[1], ld_v=hkv * hd)
        frt.frt_paged_kv_append(d)
        frt.frt_paged_kv_read(d)
        torch.cuda.synchronize()
        assert frt.frt_device_status(True) == frt.FRT_OK
        for i in range(2):
            want = v[:, i]
            if fmt == 1:
                codes, s8 = ref.quantise(want, 0.25)
                want = ref.E2M1[codes] * np.repeat(ref.E4M3[s8], 16, -1) * 0.25
            assert np.array_equal(bf16_value(runtime.bf16_host(kv[i])).reshape(want.shape), want)
        del pool


@pytest.mark.parametrize("Lq", [1, 3, 60])
@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("which", ["k_scale", "v_scale"])
def test_scales_of_nan(rt, Lq, hd, which):  # noqa: F811
    """A page scale that is NaN is not taken for a scale of nothing."""
    torch = rt[2]
    p = Problem(rt, np.random.default_rng(43), [(Lq, 150), (1, 70)], 4, 2, hd, 16)
    p.t[which].fill_(float("nan"))
    p.run()
    assert bool(torch.isnan(p.out[:p.cu[-1], :4 * hd]).all())
    assert bool(torch.isnan(p.lse[:p.cu[-1]]).all()) == (which == "k_scale")


@pytest.mark.parametrize("rows", [5, 2500])
@pytest.mark.parametrize("fmt", [0, 1])
def test_heads_without_positions_or_q(rt, rows, fmt):  # noqa: F811
    """positions NULL: 0, 1, 2, ...; an append with q_out NULL writes the
    same pages and no q; a NULL k_out or v_out is left out of a read."""
    frt, runtime, torch = rt
    case = (rows, 6, 2, 64, 32, True, True, 0)
    d, keep, q, k, _, xv = run_heads(rt, np.random.default_rng(44), *case)
    keep[2].copy_(torch.arange(rows, dtype=torch.int32))
    f, slots, pool, kv, keep2 = page_fields(rt, fmt, np.random.default_rng(45), rows, 2, 64, 16)
    for key, val in f.items():
        setattr(d, key, frt.ptr(val) if hasattr(val, "data_ptr") else val)
    frt.frt_qk_norm_rope(d)
    frt.frt_paged_kv_append(d)
    torch.cuda.synchronize()
    want = q.clone(), k.clone(), pool.clone()
    tab, pos = keep[1].cpu().numpy(), np.arange(rows)
    w = [bf16_value(runtime.bf16_host(t)).astype(np.float64) for t in keep[3:5]]
    check_rows(runtime, q, rows, 6, 64, ref.norm_rotate(xv[:, :6], w[0], 1e-6, tab, pos, 32, True))
    check_rows(runtime, k, rows, 2, 64, ref.norm_rotate(xv[:, 6:8], w[1], 1e-6, tab, pos, 32, True))
    d.positions = None
    for t in (q, k):
        t.fill_(3.0)
    pool.fill_(0xA5)
    frt.frt_qk_norm_rope(d)
    frt.frt_paged_kv_append(d)
    torch.cuda.synchronize()
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(pool, want[2])
    q.fill_(3.0)
    pool.fill_(0xA5)
    d.q_out = None
    frt.frt_paged_kv_append(d)
    torch.cuda.synchronize()
    assert bool((q == 3).all()) and torch.equal(pool, want[2])
    got = []
    for ko, vo in ((0, 1), (0, None), (None, 1)):
        for t in kv:
            t.fill_(3.0)
        d.k_out, d.ld_k = None if ko is None else frt.ptr(kv[0]), 128
        d.v_out, d.ld_v = None if vo is None else frt.ptr(kv[1]), 128
        frt.frt_paged_kv_read(d)
        torch.cuda.synchronize()
        got.append([t.clone() for t in kv])
    assert torch.equal(got[0][0], got[1][0]) and bool((got[1][1] == 3).all())
    assert torch.equal(got[0][1], got[2][1]) and bool((got[2][0] == 3).all())
    assert not bool((got[0][0] == 3).all()) and frt.frt_device_status(True) == frt.FRT_OK


@pytest.mark.parametrize("a,b", [(1, 1), (1, 60), (60, 60)])
def test_two_calls_at_once(rt, a, b):  # noqa: F811
    """Two streams, a workspace each, in turn and captured: the same bits as
    alone."""
    frt, runtime, torch = rt
    ps = [Problem(rt, np.random.default_rng(46 + i), [(n, 3000), (n, 700)], 8, 2, 128, 32) for i, n in enumerate((a, b))]
    for p in ps:
        p.run()
        p.check()
    want = [(p.out.clone(), p.lse.clone()) for p in ps]
    streams = [torch.cuda.Stream() for _ in ps]
    graphs = []
    for p, s in zip(ps, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            for _ in range(3):
                frt.frt_paged_attention_fp4(p.d)
        graphs.append(g)
    for captured in (False, True):
        for p in ps:
            p.out.fill_(5.0)
            p.lse.fill_(5.0)
        torch.cuda.synchronize()
        for _ in range(20):
            for p, s, g in zip(ps, streams, graphs):
                with torch.cuda.stream(s):
                    g.replay() if captured else frt.frt_paged_attention_fp4(p.d)
        torch.cuda.synchronize()
        assert frt.frt_device_status(True) == frt.FRT_OK
        for p, (out, lse) in zip(ps, want):
            assert torch.equal(p.out, out) and torch.equal(p.lse, lse)
            counters_are_zero(p)
