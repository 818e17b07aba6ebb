"""Every class of tiles, ranges and epilogues that the dense layers' calls of
ordinary sizes go through (dense_plans) is one that a test runs: the lists of
test_dense_gpu, and here those which these do not reach."""
import math
import random

import pytest
import torch

import dense_bounds as bounds
import dense_plans as plans
import dense_rms as rms
import sparse_mixture_experts_50_amd as moe
import test_dense_gpu as sizes
from parity import device

# type, rows, N (d), K (d_ff), activation.  By class: the gradient of h in
# ranges (every reader of its planes: streamed, small and large tiles, planes
# joined), pre-activations' gradients of every height, parity and number of
# panels, in ranges and with lower last columns, and weights' gradients of
# one, two and three matrices with and without rows behind the last stage.
GRAD = [
    ("f32", 17, 64, 64, "swiglu"), ("bf16", 18, 64, 64, "swiglu"),
    ("bf16", 19, 64, 64, "gelu"), ("f32", 21, 64, 64, "gelu"),
    ("f32", 34, 64, 64, "swiglu"), ("f32", 384, 64, 64, "gelu"),
    ("bf16", 704, 128, 64, "swiglu"), ("bf16", 832, 128, 64, "gelu"),
    ("bf16", 436, 9600, 64, "swiglu"), ("bf16", 593, 6784, 128, "swiglu"),
    ("bf16", 320, 2368, 1728, "swiglu"), ("bf16", 576, 64, 15872, "gelu"),
    ("bf16", 2505, 128, 3328, "none"), ("bf16", 4814, 1728, 128, "gelu"),
    ("f32", 1792, 704, 1536, "gelu"), ("bf16", 558, 15616, 128, "gelu"),
    ("bf16", 327, 13376, 384, "swiglu"), ("f32", 65, 8704, 1664, "gelu"),
    ("bf16", 268, 1600, 5248, "none"), ("bf16", 529, 256, 16000, "swiglu"),
    ("bf16", 2337, 4480, 384, "swiglu"), ("bf16", 2138, 512, 5120, "swiglu"),
    ("bf16", 377, 3008, 5120, "swiglu"), ("bf16", 3392, 1280, 1792, "swiglu"),
    ("bf16", 1561, 704, 6656, "swiglu"), ("bf16", 73, 10368, 4224, "swiglu"),
    ("bf16", 1536, 13760, 512, "gelu"), ("bf16", 3008, 2048, 2176, "none"),
    ("bf16", 1088, 2048, 6016, "gelu"), ("bf16", 131, 12992, 4096, "gelu"),
    ("bf16", 3476, 640, 5888, "gelu"), ("bf16", 73, 10112, 11136, "none"),
    ("bf16", 128, 11456, 14080, "gelu")]
BLOCK = [
    ("bf16", 17, 64, 64, "swiglu"), ("f32", 17, 64, 64, "gelu"),
    ("f32", 17, 64, 64, "swiglu"), ("bf16", 18, 64, 64, "gelu"),
    ("bf16", 33, 64, 64, "swiglu"), ("f32", 34, 64, 64, "swiglu"),
    ("f32", 49, 64, 64, "gelu"), ("bf16", 51, 64, 64, "gelu"),
    ("f32", 1, 448, 64, "gelu"), ("f32", 17, 448, 64, "swiglu"),
    ("f32", 26, 448, 64, "gelu"), ("f32", 33, 448, 64, "gelu"),
    ("f32", 33, 448, 64, "swiglu"), ("f32", 51, 512, 64, "gelu"),
    ("bf16", 1, 1472, 64, "swiglu"), ("bf16", 2, 1472, 64, "gelu"),
    ("bf16", 677, 64, 64, "swiglu"), ("bf16", 17, 1472, 64, "gelu"),
    ("bf16", 17, 1536, 64, "swiglu"), ("bf16", 33, 1536, 64, "gelu"),
    ("bf16", 37, 1472, 64, "swiglu"), ("bf16", 52, 1472, 64, "gelu"),
    ("bf16", 54, 1472, 64, "swiglu"), ("f32", 512, 448, 64, "swiglu"),
    ("f32", 576, 448, 64, "gelu"), ("f32", 2, 384, 5504, "swiglu"),
    ("bf16", 1216, 1664, 64, "swiglu"), ("f32", 64, 1216, 1728, "swiglu"),
    ("bf16", 712, 64, 5696, "swiglu"), ("bf16", 797, 64, 5120, "swiglu"),
    ("bf16", 268, 64, 14528, "swiglu"), ("f32", 69, 896, 4544, "swiglu"),
    ("bf16", 899, 128, 4480, "swiglu"), ("bf16", 128, 3776, 1088, "swiglu"),
    ("f32", 2240, 1024, 384, "swiglu"), ("bf16", 2409, 64, 3392, "gelu"),
    ("bf16", 1088, 64, 8064, "gelu"), ("f32", 2617, 256, 1472, "swiglu"),
    ("bf16", 333, 256, 12800, "swiglu"), ("bf16", 6546, 128, 1216, "gelu"),
    ("bf16", 551, 14720, 128, "gelu"), ("bf16", 448, 256, 11712, "swiglu"),
    ("bf16", 561, 128, 15808, "gelu"), ("bf16", 558, 192, 16256, "gelu"),
    ("f32", 3456, 2880, 256, "gelu"), ("f32", 75, 1792, 12608, "swiglu"),
    ("bf16", 4416, 2432, 320, "swiglu"), ("bf16", 1347, 384, 7488, "swiglu"),
    ("bf16", 72, 3968, 8384, "swiglu"), ("f32", 2029, 3328, 832, "swiglu"),
    ("bf16", 1625, 5312, 640, "swiglu"), ("bf16", 404, 5376, 2496, "swiglu"),
    ("bf16", 74, 12672, 3584, "swiglu"), ("bf16", 1396, 5376, 832, "swiglu"),
    ("bf16", 272, 5632, 3712, "swiglu"), ("bf16", 146, 6016, 5568, "swiglu"),
    ("bf16", 2816, 6144, 384, "swiglu"), ("bf16", 207, 4736, 8256, "swiglu"),
    ("bf16", 5756, 4864, 320, "gelu"), ("bf16", 384, 4480, 5568, "gelu"),
    ("bf16", 865, 4992, 2752, "gelu"), ("bf16", 74, 10496, 8448, "gelu"),
    ("bf16", 1427, 3840, 3008, "swiglu"), ("bf16", 321, 4608, 11008, "swiglu"),
    ("bf16", 1088, 4096, 4288, "swiglu"), ("f32", 215, 6016, 14528, "swiglu"),
    ("bf16", 401, 7488, 9536, "swiglu"), ("bf16", 2601, 8512, 1664, "swiglu"),
    ("bf16", 518, 10688, 7360, "swiglu"),
    ("bf16", 3136, 15552, 1024, "swiglu"),
    ("bf16", 7874, 5120, 2368, "swiglu")]

OTHER = {"gelu": "silu", "swiglu": "geglu"}


def reached():
    out = set()
    both = ("bf16", "f32")
    for c in [(t, *c) for c in sizes.LINEAR for t in both] + \
            sizes.LARGE + sizes.FEW:
        out |= plans.linear(*c)
    for c in [(t, *c) for c in sizes.LINEAR_GRAD for t in both] + \
            sizes.LARGE_GRAD + sizes.FEW + GRAD:
        out |= plans.linear_grad(*c)
    for c in [(t, *c) for c in sizes.DENSE + sizes.DENSE_LARGE
              for t in both] + BLOCK:
        out |= plans.dense(*c)
    return out


def test_lists_reach_every_class():
    """Of 60000 calls of up to 8192 rows and widths of up to 16384."""
    rng = random.Random(1)

    def spread(low, high):
        return int(round(math.exp(rng.uniform(math.log(low),
                                              math.log(high)))))

    have, found = reached(), {}
    for _ in range(60000):
        dtype, M = rng.choice(["bf16", "f32"]), spread(1, 8192)
        N, K = 64 * spread(1, 256), 64 * spread(1, 256)
        if rng.random() < 0.3:
            M = max(64, M // 64 * 64)
        if M * N * K > (4e11 if dtype == "bf16" else 1e11):
            continue
        call = rng.choice([plans.linear, plans.linear_grad, plans.dense])
        act = rng.choice(["none", "gelu", "swiglu"])
        if call is plans.dense and act == "none":
            act = "gelu"
        for c in call(dtype, M, N, K, act):
            found.setdefault(c, (call.__name__, dtype, M, N, K, act))
    missing = {c: s for c, s in found.items() if c not in have}
    assert not missing, f"{len(missing)} of {len(found)}: {missing}"
    assert len(found) > 250


def check(got, want, dtype, rounds, names):
    """want: (bounds, variances or None) of the outputs."""
    half = bounds.HALF[sizes.DT[dtype]]
    for n in names:
        bounds.check(got[n], want[0][n], half, rounds, n)
        if want[1] is not None:
            rms.check(got[n], want[1][n], n)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,M,N,K,act", GRAD)
def test_linear_grad(dtype, M, N, K, act):
    half = bounds.HALF[sizes.DT[dtype]]
    for a in (act, OTHER[act]) if act != "none" else (act,):
        desc, t = sizes.linear_case(dtype, M, N, K, a, True, True, seed=7)
        names = [n for n in ("x", "w", "b", "w3", "b3")
                 if n in ("x", "w", "b") or t["w3"] is not None]
        g = moe.LinearGrads(desc, device(), **{
            n: sizes.nan_like(t[n].shape, sizes.DT[dtype]) for n in names})
        moe.moe_linear_grad(desc, t["x"], sizes.weights(t), t["dy"], g,
                            sizes.workspace(
                                moe.moe_linear_grad_workspace_size(desc)),
                            dx_add=t["dx_add"])
        args = [sizes.f64(t[n]) for n in ("x", "w", "b", "w3", "b3", "dy",
                                          "dx_add")]
        check(g.as_dict(), (bounds.linear_grad(a, half, *args),
                            rms.linear_grad(a, *args) if dtype == "f32"
                            else None), dtype, 1 if a == "none" else 2, names)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,T,d,F,act", BLOCK)
def test_block(dtype, T, d, F, act):
    half = bounds.HALF[sizes.DT[dtype]]
    for a in (act, OTHER[act]):
        t, layer = sizes.dense_case(dtype, T, d, F, a, True, seed=7)
        args = [sizes.f64(t[n]) for n in sizes.OF_BLOCK]
        res, dy = sizes.f64(t["res"]), sizes.f64(t["dy"])
        y = layer.forward(t["x"], residual=t["res"])
        check({"y": y}, ({"y": bounds.dense(a, half, *args, res)},
                         {"y": rms.dense(a, *args, res)} if dtype == "f32"
                         else None), dtype, 2, ["y"])
        g = layer.backward(t["x"], t["dy"], residual=True).as_dict()
        check(g, (bounds.dense_grad(a, half, *args, dy, dy),
                  rms.dense_grad(a, *args, dy, dy) if dtype == "f32"
                  else None), dtype, 2, list(g))
        del t, layer, args, res, dy, y, g
        torch.cuda.empty_cache()
