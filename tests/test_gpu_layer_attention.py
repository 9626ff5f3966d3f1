"""The AdaRMS layer loop with attention over 4-bit pages (stack.py,
attention="paged_fp4"): the last layer's rotation, pages and attention held
to 64-bit forms on the GPU's own q/k/v, the same bits from a captured graph,
and a changed prefix changing the result."""

import numpy as np
import pytest

import paged_ref as ref
from fp8_transformer_block_b200 import synth
from fp8_transformer_block_b200.synth import bf16_value

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rt():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from fp8_transformer_block_b200 import build
    build.build()
    from fp8_transformer_block_b200 import frt, runtime, stack
    return frt, runtime, stack, torch


def workload(B, M, P, hkv, hd):
    return synth.Workload("attending", 41, "full", B=B, M=M, D=512, hq=512 // hd, hkv=hkv, hd=hd, P=P, T=P + M,
                          H=1024, layers=2, cal_rows=64)


@pytest.mark.parametrize("B,M,P,hkv,hd", [(2, 20, 37, 1, 64), (1, 50, 816, 2, 128), (3, 1, 5, 2, 64),
                                          (1, 40, 0, 1, 256)])
def test_layers_attend(rt, B, M, P, hkv, hd):
    frt, runtime, stack, torch = rt
    w = workload(B, M, P, hkv, hd)
    layers = [synth.full_layer_inputs(w, l) for l in range(w.layers)]
    x = synth.adarms_inputs(w.rows, w.D, w.seed)["res"]
    st = stack.AdaRmsLayerStack(w, layers, synth.final_norm_rows(w), x=x, attention="paged_fp4")
    st.load(x)
    st.step()
    torch.cuda.synchronize()
    assert frt.frt_device_status(True) == frt.FRT_OK
    out = st.out.clone()
    assert bool(torch.isfinite(out.float()).all())

    hq, L, a, sc = w.hq, P + M, st.att, st.scales[-1]
    qkv = bf16_value(runtime.bf16_host(a["qkv"])).reshape(w.rows, hq + 2 * hkv, hd)
    tab = a["rope"].cpu().numpy()
    pos = np.tile(np.arange(M), B)
    want_tab, ang = ref.table(M, hd, P, w.theta, 0)
    # one rounding to fp32, and the fp64 angle's own error
    assert np.all(np.abs(tab - want_tab) <= ref.F32 * np.abs(want_tab) + 16 * 2.0 ** -53 * (np.repeat(ang, 2, 1) + 1))
    q = bf16_value(runtime.bf16_host(st.q)).reshape(w.rows, hq, hd).astype(np.float64)
    v, size = ref.norm_rotate(qkv[:, :hq], None, 0, tab, pos, hd, False)
    assert np.all(np.abs(q - v) <= ref.HALF_BF16 * np.abs(v) + 10 * ref.F32 * size)

    # the pages: v and the prefix exactly, k by its distance to the rotated key
    pool = a["pool"][-1].cpu().numpy()
    pages = a["pages"].cpu().numpy()
    half, ps = pool.shape[-1] // 2, st.PAGE
    att = bf16_value(runtime.bf16_host(a["out"])).reshape(B, M, hq, hd).astype(np.float64)
    for b in range(B):
        j = np.arange(L)
        kv = []
        for i, s in ((0, sc["a_k"]), (1, sc["a_v"])):
            part = pool[..., i * half:(i + 1) * half]
            c = part[..., :ps * hd // 2].reshape(-1, hkv, ps, hd // 2)[pages[b, j // ps], :, j % ps]
            z = part[..., ps * hd // 2:].reshape(-1, hkv, ps, hd // 16)[pages[b, j // ps], :, j % ps]
            code = np.empty((L, hkv, hd), np.int64)
            code[..., 0::2], code[..., 1::2] = c & 15, c >> 4
            kv.append((ref.E2M1[code] * np.repeat(ref.E4M3[z], 16, -1) * np.float32(s)).transpose(1, 0, 2))
            rows = qkv[b * M:(b + 1) * M, hq + i * hkv:hq + (i + 1) * hkv]
            if i == 1:
                cc, ss = ref.quantise(rows, s)
                assert np.array_equal(code[P:], cc) and np.array_equal(z[P:], ss)
            else:
                key, _ = ref.norm_rotate(rows, None, 0, tab, np.arange(M), hd, False)
                got = kv[0].transpose(1, 0, 2)[P:]
                big = np.abs(key).reshape(M, hkv, -1, 16).max(-1).repeat(16, -1)
                # a code is half a step off at most: 1 of 6 (between 4 and 6)
                # of the block's largest, whose scale is within 2^-4 of it (and
                # at least half the least scale: 2^-10 of the static one); the
                # key's own bf16 rounding
                assert np.all(np.abs(got - key) <= big * (1 + 2.0 ** -4) / 6 + 6 * 2.0 ** -10 * s +
                              2 * ref.HALF_BF16 * big)
            if P:
                host = bf16_value(np.asarray(layers[-1]["prefix_k" if i == 0 else "prefix_v"]))[b]  # [hkv, P, hd]
                host = host.transpose(1, 0, 2)
                if i == 0:
                    host = np.stack([host[..., :hd // 2], host[..., hd // 2:]], -1).reshape(P, hkv, hd)
                cc, ss = ref.quantise(host, s)
                assert np.array_equal(code[:P], cc) and np.array_equal(z[:P], ss)
        want, _, tol, _ = ref.attention(q[b * M:(b + 1) * M], kv[0], kv[1], L, False, 0, hd ** -0.5)
        assert np.all(np.abs(att[b] - want) <= ref.HALF_BF16 * np.abs(want) + tol)

    # the same bits from a captured step
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        st.step()
    for _ in range(2):
        st.load(x)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, st.out)


def test_unknown_attention_is_refused(rt):
    frt, runtime, stack, torch = rt
    w = workload(1, 4, 0, 1, 64)
    layers = [synth.full_layer_inputs(w, l) for l in range(w.layers)]
    with pytest.raises(AssertionError):
        stack.AdaRmsLayerStack(w, layers, synth.final_norm_rows(w), x=None, attention="dense")


@pytest.mark.parametrize("attention", [None, "paged_fp4"])
def test_a_changed_prefix_changes_the_result(rt, attention):
    """load_prefix, eagerly and under a captured step, against a stack built
    with that prefix."""
    frt, runtime, stack, torch = rt
    w = workload(2, 20, 37, 2, 64)
    layers = [synth.full_layer_inputs(w, l) for l in range(w.layers)]
    x = synth.adarms_inputs(w.rows, w.D, w.seed)["res"]
    fin = synth.final_norm_rows(w)
    st = stack.AdaRmsLayerStack(w, layers, fin, x=x, attention=attention)
    changed = []
    for l, ly in enumerate(layers):
        k, v = np.asarray(ly["prefix_k"]), np.asarray(ly["prefix_v"])
        # other tokens of the same sizes: turned around, signs changed
        changed.append(dict(ly, prefix_k=np.ascontiguousarray(k[:, :, ::-1]) ^ 0x8000,
                            prefix_v=np.ascontiguousarray(v[:, :, ::-1])))
    other = stack.AdaRmsLayerStack(w, changed, fin, scales=st.scales, attention=attention)

    def result(run, s):
        s.load(x)
        run()
        torch.cuda.synchronize()
        return [s.out.clone()] + [s.lay[l][c][:, :w.P].clone() for l in range(w.layers) for c in ("kc", "vc")]

    first, want = result(st.step, st), result(other.step, other)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        st.step()
    st.load_prefix([(ly["prefix_k"], ly["prefix_v"]) for ly in changed])
    for run in (st.step, graph.replay):
        got = result(run, st)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        # the stand-in's result does not hang on the prefix, its caches do
        assert not torch.equal(got[1], first[1])
        assert torch.equal(got[0], first[0]) == (attention is None)
    st.load_prefix([(ly["prefix_k"], ly["prefix_v"]) for ly in layers])
    assert all(torch.equal(a, b) for a, b in zip(result(graph.replay, st), first))
    with pytest.raises(AssertionError):
        st.load_prefix([(changed[0]["prefix_k"], changed[0]["prefix_v"])])
    with pytest.raises(AssertionError):
        st.load_prefix([(ly["prefix_k"][:, :, 1:], ly["prefix_v"]) for ly in layers])
