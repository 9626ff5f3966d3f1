"""GPU parity of the attention over 4-bit pages against a 64-bit form,
through the C ABI: head layouts, lengths, masks, pages and index errors, and
the cache's operators run together."""

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


class Problem:
    """Sequences of (query rows, keys) over a shuffled pool whose unused
    bytes are all 0xFF (NaN scales)."""

    def __init__(self, rt, rng, lens, hq, hkv, hd, ps, causal=True, window=0, pad=0, spare_rows=3, lse=True,
                 q_gain=1.0, scale=None, extra_pages=0):
        frt, runtime, torch = self.rt = rt
        self.lens, self.hq, self.hkv, self.hd, self.ps = lens, hq, hkv, hd, ps
        self.causal, self.window, self.scale = causal, window, hd ** -0.5 if scale is None else scale
        n = len(lens)
        need = [(L + ps - 1) // ps for _, L in lens]
        self.max_pages = max(max(need), 1) + extra_pages
        self.n_pages = sum(need) + 2
        ids = rng.permutation(self.n_pages)[:sum(need)]
        self.table = np.full((n, self.max_pages), -7, np.int32)
        pool = np.full((self.n_pages, hkv, frt.frt_kv_record_bytes(1, ps, hd)), 0xFF, np.uint8)
        half = pool.shape[-1] // 2
        self.ks, self.vs = np.float32(0.0371), np.float32(0.25)
        self.kv = []
        at = 0
        for s, (_, L) in enumerate(lens):
            pages = ids[at:at + need[s]]
            at += need[s]
            self.table[s, :need[s]] = pages
            both = []
            for i, static in ((0, self.ks), (1, self.vs)):
                codes = rng.integers(0, 256, (L, hkv, hd // 2), dtype=np.uint8)
                sc = rng.integers(0x30, 0x48, (L, hkv, hd // 16), dtype=np.uint8)
                j = np.arange(L)
                part = pool[..., i * half:(i + 1) * half]
                c = part[..., :ps * hd // 2].reshape(self.n_pages, hkv, ps, hd // 2)
                z = part[..., ps * hd // 2:].reshape(self.n_pages, hkv, ps, hd // 16)
                c[pages[j // ps], :, j % ps], z[pages[j // ps], :, j % ps] = codes, sc
                part[..., :ps * hd // 2] = c.reshape(self.n_pages, hkv, -1)
                part[..., ps * hd // 2:] = z.reshape(self.n_pages, hkv, -1)
                x = np.empty((L, hkv, hd))
                x[..., 0::2], x[..., 1::2] = ref.E2M1[codes & 15], ref.E2M1[codes >> 4]
                both.append((x * np.repeat(ref.E4M3[sc], 16, -1) * static).transpose(1, 0, 2))
            self.kv.append(both)
        self.cu = np.zeros(n + 1, np.int32)
        self.cu[1:] = np.cumsum([q for q, _ in lens])
        self.rows = int(self.cu[-1]) + spare_rows
        qf = rng.standard_normal((self.rows, hq * hd + pad), dtype=np.float32) * q_gain
        self.q = bf16_bits(qf)
        dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        self.t = dict(q=runtime.bf16_dev(self.q), pool=dev(pool), page_table=dev(self.table), cu_rows=dev(self.cu),
                      kv_len=dev(np.array([L for _, L in lens], np.int32)), k_scale=runtime.scale_dev(self.ks),
                      v_scale=runtime.scale_dev(self.vs))
        self.out = torch.full((self.rows, hq * hd + pad), 5.0, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((self.rows, hq), 5.0, device="cuda") if lse else None
        max_q = max(1, max(q for q, _ in lens))
        self.nbytes = frt.frt_paged_attention_workspace_size(n, max_q, hq, hkv, hd)
        self.ws = runtime.workspace(self.nbytes)
        self.counters = self.nbytes > 0   # the head of the workspace holds counters
        self.d = runtime.paged_attn_desc(
            n_seqs=n, rows=self.rows, max_q=max_q, hq=hq, hkv=hkv, hd=hd, page_size=ps, max_pages=self.max_pages,
            n_pages=self.n_pages, causal=int(causal), window=window, sm_scale=self.scale, ld_q=hq * hd + pad,
            ld_out=hq * hd + pad, out=self.out, lse=self.lse, workspace=self.ws, workspace_bytes=self.nbytes, **self.t)

    def run(self, stream=None, report=True):
        frt, runtime, torch = self.rt
        frt.frt_paged_attention_fp4(self.d, stream=stream)
        torch.cuda.synchronize()
        if report:
            assert frt.frt_device_status(True) == frt.FRT_OK

    def results(self):
        frt, runtime, torch = self.rt
        o = bf16_value(runtime.bf16_host(self.out)).astype(np.float64)
        return o, None if self.lse is None else self.lse.cpu().numpy().astype(np.float64)

    def check(self, only=None, kv=None):
        frt, runtime, torch = self.rt
        o, lse = self.results()
        w = self.hq * self.hd
        qv = bf16_value(self.q)[:, :w].astype(np.float64)
        for s, (Lq, L) in enumerate(self.lens):
            if only is not None and s not in only:
                continue
            lo, hi = self.cu[s], self.cu[s + 1]
            k, v = (kv or self.kv)[s]
            want, wl, tol, tl = ref.attention(qv[lo:hi].reshape(Lq, self.hq, self.hd), k, v, L, self.causal,
                                              self.window, self.scale)
            got = o[lo:hi, :w].reshape(want.shape)
            err = np.abs(got - want) - (ref.HALF_BF16 * np.abs(want) + tol)
            assert not err.size or err.max() <= 0, (s, Lq, L, float(err.max()))
            if lse is not None:
                g = lse[lo:hi]
                empty = np.isneginf(wl)
                assert np.array_equal(np.isneginf(g), empty)
                assert np.all(np.abs(g[~empty] - wl[~empty]) <= tl[~empty])
        assert np.all(o[self.cu[-1]:] == 5.0) and np.all(o[:, w:] == 5.0)
        assert lse is None or np.all(lse[self.cu[-1]:] == 5.0)
        if self.counters:
            assert int(self.ws[:4 * 148].view(torch.int32).abs().sum()) == 0


LENGTHS = [1, 2, 15, 16, 17, 31, 63, 64, 65, 127, 128, 129, 255, 257, 500, 1025]


@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 1), (8, 2), (6, 3), (7, 1), (16, 1), (40, 2)])
def test_single_tokens(rt, hd, hq, hkv):
    rng = np.random.default_rng(hd + hq)
    p = Problem(rt, rng, [(1, L) for L in LENGTHS], hq, hkv, hd, 16 if hd == 256 else 32)
    p.run()
    p.check()
    assert rt[0].frt_device_status(True) == 0


@pytest.mark.parametrize("ps", [16, 32, 64, 128, 512, 1024])
@pytest.mark.parametrize("causal,window", [(False, 0), (True, 0), (True, 37)])
def test_pages_and_masks(rt, ps, causal, window):
    rng = np.random.default_rng(ps + causal)
    lens = [(1, 1), (3, 3), (5, 64), (1, 1300), (0, 40), (9, 700), (2, 2), (13, 130)]
    p = Problem(rt, rng, lens, 4, 2, 64, ps, causal, window, pad=8, extra_pages=2)
    p.run()
    p.check()


@pytest.mark.parametrize("hd,hq,hkv", [(64, 8, 1), (128, 4, 4), (128, 32, 8), (256, 8, 1), (256, 2, 2)])
@pytest.mark.parametrize("causal,window", [(False, 0), (True, 0), (True, 100)])
def test_many_query_rows(rt, hd, hq, hkv, causal, window):
    rng = np.random.default_rng(hd + hq + causal)
    p = Problem(rt, rng, [(50, 866), (1, 200), (129, 129), (0, 0), (77, 300), (257, 1000)], hq, hkv, hd, 64, causal,
                window)
    p.run()
    p.check()


def test_rows_that_see_no_key(rt):
    """No keys at all, and more queries than keys under the causal mask."""
    rng = np.random.default_rng(7)
    for hd in (64, 128, 256):
        p = Problem(rt, rng, [(3, 0), (1, 0), (9, 4), (40, 1), (1, 5)], 8, 2, hd, 16)
        p.run()
        p.check()
        o, lse = p.results()
        assert np.all(o[:4, :8 * hd] == 0) and np.all(np.isneginf(lse[:4]))


@pytest.mark.parametrize("n", [159, 160, 161, 700])
def test_many_sequences(rt, n):
    rng = np.random.default_rng(n)
    lens = [(int(rng.integers(0, 3)), int(rng.integers(0, 90))) for _ in range(n)]
    lens[-1] = (1, 33)
    p = Problem(rt, rng, lens, 4, 1, 64, 16)
    p.run()
    p.check()


def test_peaked_and_far_scores(rt):
    """Scores far apart (the running maximum moves by hundreds), far below
    and above zero, a negative scale, and rows of tiny and huge q."""
    rng = np.random.default_rng(8)
    p = Problem(rt, rng, [(4, 400), (1, 900)], 8, 1, 128, 32, q_gain=30.0)
    p.run()
    p.check()
    p = Problem(rt, rng, [(4, 400), (1, 900)], 8, 1, 128, 32, scale=-0.3)
    p.run()
    p.check()
    for gain in (2.0 ** -100, 2.0 ** 60):
        p = Problem(rt, rng, [(2, 100)], 8, 1, 64, 32, q_gain=gain, scale=0.125 / gain)
        p.run()
        p.check()


@pytest.mark.parametrize("window", [2 ** 30, 2 ** 31 - 40, 2 ** 31 - 1])
@pytest.mark.parametrize("Lq", [6, 300])
def test_windows_past_every_key(rt, Lq, window):
    """The largest windows hide nothing, also where a tile's first queries
    stand before the first key."""
    p = Problem(rt, np.random.default_rng(21), [(Lq, 5), (Lq, 200), (1, 77)], 8, 2, 64, 16, window=window)
    p.run()
    p.check()


@pytest.mark.parametrize("Lq", [1, 60])
def test_scale_of_zero(rt, Lq):
    """Every visible key weighs the same."""
    p = Problem(rt, np.random.default_rng(20), [(Lq, 150), (1, 70)], 4, 2, 64, 16, scale=0.0)
    p.run()
    p.check()


def test_one_long_sequence(rt):
    rng = np.random.default_rng(9)
    p = Problem(rt, rng, [(1, 40000)], 8, 2, 128, 64)
    p.run()
    p.check()
    first = p.out.clone()
    for _ in range(3):   # the same bits from call to call
        p.out.fill_(5.0)
        p.run()
        import torch
        assert torch.equal(first, p.out)


def test_no_lse_and_uniform_rows(rt):
    """cu_rows NULL: max_q rows each; lse NULL."""
    rng = np.random.default_rng(10)
    p = Problem(rt, rng, [(3, 50), (3, 200), (3, 3)], 4, 2, 64, 16, lse=False, spare_rows=0)
    p.d.cu_rows = None
    p.run()
    p.check()


@pytest.mark.parametrize("max_q", [1, 200])
def test_indices_out_of_range(rt, max_q):
    """A bad page hides its tokens, a long length is held to the table, rows
    to the tensor and to max_q; each is reported, none is followed."""
    frt, runtime, torch = rt
    rng = np.random.default_rng(11)
    Lq = max_q
    p = Problem(rt, rng, [(Lq, 600), (Lq, 300)], 4, 1, 64, 64, causal=False)
    for bad in (-1, p.n_pages, 2 ** 31 - 1):
        p.t["page_table"][0, 3] = bad
        p.run(report=False)
        assert frt.frt_device_status(True) == frt.FRT_ERANGE
        keep = np.r_[0:192, 256:600]
        k, v = p.kv[0]
        want, wl, tol, tl = ref.attention(bf16_value(p.q)[:Lq].astype(np.float64).reshape(Lq, 4, 64), k[:, keep],
                                          v[:, keep], len(keep), False, 0, p.scale)
        got = p.results()[0][:Lq].reshape(want.shape)
        assert np.all(np.abs(got - want) <= ref.HALF_BF16 * np.abs(want) + tol)
        p.check(only=[1])
    p.t["page_table"].copy_(torch.from_numpy(p.table))
    p.run(report=False)
    assert frt.frt_device_status(True) == frt.FRT_OK
    p.check()
    p.t["kv_len"][1] = -5
    p.run(report=False)
    assert frt.frt_device_status(True) == frt.FRT_ERANGE
    o, lse = p.results()
    assert np.all(o[Lq:2 * Lq] == 0) and np.all(np.isneginf(lse[Lq:2 * Lq]))
    p.check(only=[0])
    p.t["kv_len"][1] = 300
    for cu in ([0, Lq, 5 * Lq + 99], [-4, Lq, 2 * Lq], [0, Lq, 0]):
        p.t["cu_rows"].copy_(torch.tensor(cu, dtype=torch.int32))
        p.out.fill_(5.0)
        p.lse.fill_(5.0)
        p.run(report=False)
        assert frt.frt_device_status(True) == frt.FRT_ERANGE
        p.check(only=[0]) if cu[0] == 0 and cu[1] == Lq and cu[2] > 0 else None
    p.t["cu_rows"].copy_(torch.tensor([0, Lq, 2 * Lq], dtype=torch.int32))
    p.out.fill_(5.0)
    p.lse.fill_(5.0)
    p.run(report=False)
    assert frt.frt_device_status(True) == frt.FRT_OK
    p.check()


@pytest.mark.parametrize("Lq", [1, 150])
def test_another_stream_and_a_graph(rt, Lq):
    frt, runtime, torch = rt
    rng = np.random.default_rng(12)
    p = Problem(rt, rng, [(Lq, 700), (Lq, 333)], 8, 1, 128, 32)
    p.run()
    p.check()
    want = p.out.clone()
    s = torch.cuda.Stream()
    p.out.fill_(5.0)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        frt.frt_paged_attention_fp4(p.d)
    s.synchronize()
    assert torch.equal(want, p.out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        frt.frt_paged_attention_fp4(p.d)
        frt.frt_paged_attention_fp4(p.d)
    p.out.fill_(5.0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(want, p.out)
    # new lengths under the same graph: sizes are read on the device
    p.t["kv_len"].copy_(torch.tensor([650, 200], dtype=torch.int32))
    p.lens = [(Lq, 650), (Lq, 200)]
    p.kv = [[x[:, :L] for x in kv] for kv, (_, L) in zip(p.kv, p.lens)]
    graph.replay()
    torch.cuda.synchronize()
    p.check()


@pytest.mark.parametrize("hd,rot,half", [(64, 64, True), (128, 32, False), (256, 256, True)])
def test_append_then_attend(rt, hd, rot, half):
    """Prompts of three sequences, then single tokens, through norm, rotation,
    append and attention; the reference reads the cache back."""
    frt, runtime, torch = rt
    rng = np.random.default_rng(hd)
    hq, hkv, ps, n_pages = 8, 2, 32, 40
    tab = torch.empty(512, rot, device="cuda")
    frt.frt_build_rope_table_scaled(512, rot, 0, 1e4, frt.FRT_ROPE_SCALE_LINEAR, 2.0, 0, 0, 0, 1.0, tab)
    qn = runtime.bf16_dev(bf16_bits(1 + 0.1 * rng.standard_normal(hd, dtype=np.float32)))
    pool = runtime.kv_pool(n_pages, hkv, ps, hd)
    ks, vs = runtime.scale_dev(0.01), runtime.scale_dev(0.02)
    order = rng.permutation(n_pages)
    pages = [order[:12], order[12:20], order[20:30]]
    table = np.full((3, 12), -1, np.int32)
    for s, pg in enumerate(pages):
        table[s, :len(pg)] = pg
    table_d = torch.from_numpy(table).cuda()
    have = [0, 0, 0]
    for step in ([200, 31, 97], [1, 1, 1], [1, 0, 1], [2, 1, 5]):
        rows = sum(step)
        pos, slots = [], []
        for s, nq in enumerate(step):
            for j in range(have[s], have[s] + nq):
                pos.append(j)
                slots.append(int(pages[s][j // ps]) * ps + j % ps)
            have[s] += nq
        pos.append(0)          # a padding row
        slots.append(-1)
        x = runtime.bf16_dev(bf16_bits(rng.standard_normal((rows + 1, (hq + 2 * hkv) * hd), dtype=np.float32)))
        q = runtime.empty_bf16(rows + 1, hq * hd)
        pos_d = torch.tensor(pos, dtype=torch.int32, device="cuda")
        slot_d = torch.tensor(slots, device="cuda")
        d = runtime.qk_rope_desc(
            rows=rows + 1, hq=hq, hkv=hkv, hd=hd, rot=rot, layout=int(half), eps=1e-6, qkv=x, ld_qkv=x.shape[1],
            q_norm=qn, k_norm=qn, rope=tab, n_pos=512, positions=pos_d, q_out=q, ld_q=hq * hd, format=1,
            page_size=ps, n_pages=n_pages, pool=pool, slots=slot_d, k_scale=ks, v_scale=vs)
        frt.frt_paged_kv_append(d)
        cu = torch.tensor(np.r_[0, np.cumsum(step)], dtype=torch.int32, device="cuda")
        kl = torch.tensor(have, dtype=torch.int32, device="cuda")
        out = torch.full((rows + 1, hq * hd), 5.0, dtype=torch.bfloat16, device="cuda")
        nb = frt.frt_paged_attention_workspace_size(3, max(step), hq, hkv, hd)
        ws = runtime.workspace(nb)
        frt.frt_paged_attention_fp4(runtime.paged_attn_desc(
            n_seqs=3, rows=rows, max_q=max(step), hq=hq, hkv=hkv, hd=hd, page_size=ps, max_pages=12, n_pages=n_pages,
            causal=1, window=0, sm_scale=hd ** -0.5, q=q, ld_q=hq * hd, pool=pool, page_table=table_d, cu_rows=cu,
            kv_len=kl, k_scale=ks, v_scale=vs, out=out, ld_out=hq * hd, lse=None, workspace=ws, workspace_bytes=nb))
        torch.cuda.synchronize()
        got = bf16_value(runtime.bf16_host(out)).astype(np.float64)
        qv = bf16_value(runtime.bf16_host(q)).astype(np.float64)
        pl = pool.cpu().numpy()
        lo = 0
        for s, nq in enumerate(step):
            j = np.arange(have[s])
            page, at = pages[s][j // ps], j % ps
            kv = []
            for i, sc in ((0, 0.01), (1, 0.02)):
                part = pl[..., i * pl.shape[-1] // 2:(i + 1) * pl.shape[-1] // 2]
                c = part[..., :ps * hd // 2].reshape(n_pages, hkv, ps, hd // 2)[page, :, at]
                z = part[..., ps * hd // 2:].reshape(n_pages, hkv, ps, hd // 16)[page, :, at]
                v = np.empty((len(j), hkv, hd))
                v[..., 0::2], v[..., 1::2] = ref.E2M1[c & 15], ref.E2M1[c >> 4]
                kv.append((v * np.repeat(ref.E4M3[z], 16, -1) * np.float32(sc)).transpose(1, 0, 2))
            want, _, tol, _ = ref.attention(qv[lo:lo + nq].reshape(nq, hq, hd), kv[0], kv[1], have[s], True, 0,
                                            hd ** -0.5)
            g = got[lo:lo + nq].reshape(want.shape)
            assert np.all(np.abs(g - want) <= ref.HALF_BF16 * np.abs(want) + tol)
            lo += nq
        assert np.all(got[rows] == 5.0)
    assert frt.frt_device_status(True) == frt.FRT_OK
