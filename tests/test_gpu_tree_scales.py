"""Draft-tree attention over pools with a scale per token, whose value scales lie far apart:
the result keeps its precision relative to its own terms, whatever scale a token of little
weight has."""
import numpy as np
import pytest
import torch

import workloads as W
from tests import tree_ref as T
from tests.test_gpu_tree import case, make

pytestmark = pytest.mark.gpu

BF, F8, TOKEN = W.KV_BF16, W.KV_FP8, W.SCALE_PER_TOKEN_HEAD


def check(w, c):
    """out and lse of a causal chain against 64 bits.

    Bounds, with p the weights: a logit is off by at most d = 130 * 2^-23 of the sum of its
    terms' absolute values, p by 2 d of itself; P = p * scale is rounded to 16 bits by half a
    step (f16: 2^-11, bf16: 2^-8) and the sums by 3e-5 in all, relative to a = sum p |v|; the
    result to bf16 by 2^-8 of itself.  f16 below 2^-14 rounds by 2^-25 where a row's largest P is
    2^2 or more (7 above the reference, which may be 4 too high and rests on log2 of the scales to
    0.09), so by 2^-27 of the largest p * scale, times the codes."""
    n, h, _ = w.q.shape
    q = T.values(w.q)
    got, gl = c.out.double().cpu().numpy(), c.lse.double().cpu().numpy()
    for r in range(w.num_reqs):
        ctx, q0, q1 = int(w.context_lens[r]), int(w.cu_seqlens_q[r]), int(w.cu_seqlens_q[r + 1])
        tot = ctx + q1 - q0
        pages = w.block_table[r, :(tot + 127) // 128]
        k = T._scaled(w, w.k_cache, w.k_scale, pages, tot)
        v = T._scaled(w, w.v_cache, w.v_scale, pages, tot)
        vs = np.abs(w.v_scale[pages].astype(np.float64).reshape(-1)[:tot])
        codes = np.abs(T.values(w.v_cache[pages]).reshape(-1, 128)[:tot])
        for j in range(q1 - q0):
            end = ctx + j + 1
            z = w.softmax_scale * (q[q0 + j] @ k[:end].T)
            d = (130 * 2.0 ** -23 * w.softmax_scale * (np.abs(q[q0 + j]) @ np.abs(k[:end]).T)).max(1, keepdims=True)
            lse = np.log(np.exp(z - z.max(1, keepdims=True)).sum(1, keepdims=True)) + z.max(1, keepdims=True)
            p = np.exp(z - lse)
            out, a = p @ v[:end], p @ np.abs(v[:end])
            tol = (2.0 ** (-11 if w.kv_dtype == F8 else -8) + 2 * d + 3e-5) * a + 2.0 ** -8 * np.abs(out) + 1e-30
            if w.kv_dtype == F8:
                tol += 2.0 ** -27 * (p * vs[:end]).max(1, keepdims=True) * codes[:end].sum(0)
            err = np.abs(got[q0 + j] - out)
            assert (err <= tol).all(), (r, j, (err / tol).max())
            assert (np.abs(gl[q0 + j] - lse[:, 0]) <= d[:, 0] + 2e-5 + 2.0 ** -21 * np.abs(lse[:, 0])).all()


def place(w, r, pos):
    return w.block_table[r, pos // 128], pos % 128


SHAPES = [(16, 1), (16, 2), (16, 3), (16, 20), (5, 33)]  # each kernel and tile


@pytest.mark.parametrize("kv", [BF, F8])
@pytest.mark.parametrize("hq,ql", SHAPES)
@pytest.mark.parametrize("ctx", [300, 20000])
@pytest.mark.parametrize("light,heavy", [(-20, 0), (-26, 0), (-30, 4), (0, 26), (-39, -12), (12, 39)])
@pytest.mark.parametrize("where", ["before", "behind", "beside"])
def test_a_large_scale_of_little_weight(kv, hq, ql, ctx, light, heavy, where):
    # one token has nearly all the weight (e^40 of any other's) and the scale 2^light; another one
    # has next to none and the scale 2^heavy, far before or behind it or in the same 16 tokens
    w = make(51, [ql, 1], [ctx, 200], hq, kv, TOKEN)
    w.k_scale[:] = 1
    w.v_scale[:] *= 2.0 ** light
    w.q[:, :, 0] = W.bf16_bits(np.array([8.0]))[0]
    num = (lambda x: W.fp8_codes(np.array([x]))[0]) if kv == F8 else (lambda x: W.bf16_bits(np.array([x]))[0])
    for r, n in ((0, ctx), (1, 200)):
        pages = w.block_table[r, :(n + ql + 127) // 128]
        w.k_cache[pages[pages >= 0], :, 0, 0] = num(0.0)
        one, other = {"before": (n - 9, n // 7), "behind": (n // 7, n - 9), "beside": (n - 9, (n - 9) ^ 3)}[where]
        w.k_cache[(*place(w, r, one), 0, 0)] = num(56.0)
        w.v_scale[place(w, r, one)] = 2.0 ** light
        w.v_scale[place(w, r, other)] = 2.0 ** heavy
    c = case(w)
    c.tree_attn()
    torch.cuda.synchronize()
    assert int(c.status.item()) == 0
    check(w, c)


@pytest.mark.parametrize("kv", [BF, F8])
@pytest.mark.parametrize("hq,ql", SHAPES)
def test_scales_over_many_magnitudes(kv, hq, ql):
    w = make(52, [ql, ql], [5000, 130], hq, kv, TOKEN)
    w.v_scale[:] = np.exp2(np.random.default_rng(3).uniform(-38, 38, w.v_scale.shape)) * \
        np.random.default_rng(4).choice([-1.0, 1.0], w.v_scale.shape)
    c = case(w)
    c.tree_attn()
    torch.cuda.synchronize()
    check(w, c)


@pytest.mark.parametrize("kv", [BF, F8])
@pytest.mark.parametrize("hq,ql", SHAPES)
def test_a_zero_vector_in_a_long_context(kv, hq, ql):
    # an inserted vector of zeros has the scale 1, the others' are near 0.01
    w = make(53, [ql], [30000], hq, kv, TOKEN)
    w.v_scale[:] *= 0.01
    c = case(w)
    g = torch.Generator("cuda").manual_seed(5)
    k_new, v_new, idx_new = (torch.randn((ql, 1, 128), generator=g, device="cuda").to(torch.bfloat16) for _ in range(3))
    v_new[0] = 0
    if kv == F8:
        c.kv_insert(k_new, v_new, idx_new)
        torch.cuda.synchronize()
        w.k_cache, w.v_cache = c.k.cpu().numpy(), c.v.cpu().numpy()
        w.k_scale, w.v_scale = c.k_scale.cpu().numpy(), c.v_scale.cpu().numpy()
        assert w.v_scale[place(w, 0, 30000)] == 1
    else:  # (bf16 pools take copies; their scales are the caller's)
        w.v_cache[place(w, 0, 30000)] = 0
        w.v_scale[place(w, 0, 30000)] = 1
        c = case(w)
    c.tree_attn()
    torch.cuda.synchronize()
    check(w, c)


@pytest.mark.parametrize("kv", [BF, F8])
@pytest.mark.parametrize("ql", [1, 20])
@pytest.mark.parametrize("scale", [0.0, 1e-42, 2.0 ** -126, 2.0 ** -100])
def test_scales_of_zero_and_near_it(kv, ql, scale):
    # tokens with such a scale, with most of the weight or all of them: results stay finite
    # and within a bf16 of the other tokens'
    w = make(54, [ql], [700], 16, kv, TOKEN)
    w.v_scale[w.block_table[0, 1:3]] = scale
    c = case(w)
    c.tree_attn()
    torch.cuda.synchronize()
    check(w, c)
    w.v_scale[:] = scale
    c = case(w)
    c.tree_attn()
    torch.cuda.synchronize()
    assert (c.out.float().abs() <= 448 * scale * 1.01).all()
    ref = T.tree_attn(w)
    assert (np.abs(c.lse.double().cpu().numpy() - ref[1]) <= ref[3]).all()
