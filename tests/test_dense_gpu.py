"""Linear layers, the feed-forward block and their gradients on the GPU
against float64 (dense_bounds), at the sizes where their kernels change."""
import pytest
import torch

import dense_bounds as ref
import sparse_mixture_experts_50_amd as moe
from parity import device

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
ACTS = ["none", "gelu", "silu", "swiglu", "geglu"]


def normal(g, shape, std, dtype):
    return torch.empty(shape, dtype=dtype, device=device()) \
        .normal_(0.0, std, generator=g)


def generator(seed):
    return torch.Generator(device=device()).manual_seed(seed)


def f64(t):
    return None if t is None else t.double()


def linear_case(dtype, M, N, K, act, bias, res, seed=0):
    g, dt = generator(seed + M + 7 * N + 31 * K), DT[dtype]
    gated = act in ref.GATED
    t = {"x": normal(g, (M, K), 1.0, dt),
         "w": normal(g, (N, K), K ** -0.5, dt),
         "b": normal(g, (N,), 0.5, dt) if bias else None,
         "w3": normal(g, (N, K), K ** -0.5, dt) if gated else None,
         "b3": normal(g, (N,), 0.5, dt) if bias and gated else None,
         "res": normal(g, (M, N), 1.0, dt) if res else None,
         "dy": normal(g, (M, N), 1.0, dt),
         "dx_add": normal(g, (M, K), 1.0, dt) if res else None}
    return moe.make_linear_desc(M, N, K, dt, activation=act), t


def weights(t):
    return moe.LinearWeights(t["w"], b=t["b"], w3=t["w3"], b3=t["b3"])


def workspace(n, fill=0xFF):
    """Filled with bytes that are not a number in either type."""
    return torch.full((n,), fill, dtype=torch.uint8, device=device())


def nan_like(shape, dtype):
    return torch.full(shape, float("nan"), dtype=dtype, device=device())


# Few rows: weights streamed, every count of row blocks, wide outputs with two
# and four column blocks a wave, K that the waves share unevenly or not at
# all.  More rows: small tiles with ends on both axes, ranges of K.  Many:
# large tiles of every height, an odd number of stages, more row tiles than a
# strip.
LINEAR = [
    (1, 64, 64, "none"), (1, 4096, 4096, "none"), (7, 192, 320, "gelu"),
    (16, 128, 704, "swiglu"), (17, 16384, 64, "silu"), (5, 32768, 128, "none"),
    (30, 16384, 192, "geglu"), (33, 320, 1024, "swiglu"),
    (64, 2816, 1024, "gelu"), (65, 64, 64, "none"), (65, 128, 4096, "swiglu"),
    (127, 192, 128, "silu"), (300, 64, 2048, "geglu"), (257, 448, 192, "gelu"),
    (1000, 2048, 1024, "none"), (2049, 4096, 192, "gelu"),
    (1537, 5120, 320, "swiglu"), (2300, 4160, 256, "silu"),
    (100, 65536, 128, "none"), (400, 32768, 64, "geglu"),
    (1021, 1984, 1024, "gelu"),
]


# The large tiles: of 128 to 256 rows, an odd and an even number of stages,
# whole and in ranges of K, with one and with two panels; single precision's.
LARGE = [("bf16", *c) for c in [
    (266, 6592, 4992, "none"), (1110, 7296, 512, "gelu"),
    (1095, 9088, 320, "silu"), (203, 9792, 5120, "none"),
    (4845, 3008, 128, "none"), (2282, 3648, 64, "gelu"),
    (1417, 1536, 5120, "silu"), (96, 8960, 4224, "swiglu"),
    (564, 8128, 2176, "geglu"), (558, 7808, 704, "swiglu"),
    (132, 5632, 3712, "geglu"), (822, 7936, 256, "geglu"),
    (849, 5952, 320, "swiglu"), (2670, 2112, 128, "swiglu"),
    (1012, 5504, 64, "geglu"), (256, 4288, 4992, "swiglu"),
    # (lower tiles in the last columns, or in all)
    (3308, 6336, 384, "none"), (2680, 7744, 448, "gelu"),
    (920, 6720, 2368, "silu"), (4981, 1216, 2176, "none"),
    (1177, 8832, 384, "swiglu"), (1881, 5504, 448, "geglu"),
    (1975, 1664, 2240, "swiglu")]] + [
    ("f32", *c) for c in [
        (2562, 2944, 256, "gelu"), (2984, 2432, 64, "none"),
        (4531, 768, 128, "swiglu"), (1336, 2112, 64, "geglu"),
        (1910, 4288, 128, "none"), (4216, 1600, 64, "gelu"),
        (69, 6848, 3200, "none"), (68, 4928, 5760, "silu"),
        (5075, 768, 128, "swiglu"), (362, 8960, 64, "geglu"),
        (65, 4224, 2560, "swiglu"), (67, 6400, 2240, "geglu")]]


# few rows of few columns, in ranges of K
FEW = [(t, *c) for t in ("bf16", "f32") for c in [
    (6, 64, 6976, "geglu"), (48, 64, 6976, "swiglu"), (1, 64, 19968, "gelu"),
    (45, 128, 8000, "silu"), (64, 64, 16384, "none"),
    (64, 1024, 8192, "none"), (45, 2048, 4096, "swiglu")]]


@pytest.mark.parametrize("dtype,M,N,K,act",
                         [(t, *c) for c in LINEAR for t in ("bf16", "f32")] +
                         LARGE + FEW)
def test_linear(dtype, M, N, K, act):
    half = ref.HALF[DT[dtype]]
    for bias, res in ((False, False), (True, True)):
        desc, t = linear_case(dtype, M, N, K, act, bias, res)
        y = nan_like((M, N), DT[dtype])
        moe.moe_linear(desc, t["x"], weights(t), y,
                       workspace(moe.moe_linear_workspace_size(desc)),
                       residual=t["res"])
        want = ref.linear(act, half, *(f64(t[n]) for n in (
            "x", "w", "b", "w3", "b3", "res")))
        ref.check(y, want, half, 1, f"y, bias {bias}")


LINEAR_GRAD = [
    (1, 64, 64, "none"), (1, 1024, 2048, "gelu"), (33, 2816, 1024, "gelu"),
    (16, 192, 320, "swiglu"), (63, 128, 128, "silu"), (64, 320, 64, "geglu"),
    (65, 64, 704, "none"), (130, 448, 192, "swiglu"), (1000, 64, 64, "silu"),
    (2049, 2048, 1024, "none"), (2300, 1024, 2112, "swiglu"),
    (4100, 320, 256, "gelu"), (777, 1984, 1024, "geglu"),
]


# Large tiles in the rows' gradient (of one and of two products), the weights'
# and the pre-activations computed again.
LARGE_GRAD = [("bf16", *c) for c in [
    (277, 4736, 6720, "none"), (1057, 128, 8000, "none"),
    (862, 192, 9920, "none"), (219, 4608, 8256, "none"),
    (3718, 64, 4032, "none"), (1762, 5504, 1216, "silu"),
    (83, 4992, 8960, "swiglu"), (291, 2304, 6848, "geglu"),
    (1032, 448, 8448, "swiglu"), (1487, 64, 5440, "geglu"),
    (2804, 2496, 704, "swiglu"), (77, 2624, 5120, "none"),
    (4242, 1728, 1600, "none"), (4137, 960, 1408, "swiglu"),
    (1110, 7296, 512, "gelu"), (1095, 9088, 320, "silu"),
    (2282, 3648, 64, "gelu"), (558, 7808, 704, "swiglu"),
    (2670, 2112, 128, "geglu"), (1012, 5504, 64, "swiglu"),
    # (lower tiles in the last columns, or in all)
    (1881, 5504, 448, "swiglu"), (2680, 7744, 448, "silu"),
    (2875, 384, 7296, "none"), (6583, 448, 3136, "none"),
    (6209, 2368, 960, "none"), (2197, 192, 9600, "swiglu"),
    (2745, 1088, 2368, "geglu")]] + [
    ("f32", 993, 64, 6208, "none"), ("f32", 2562, 2944, 256, "silu"),
    ("f32", 1336, 2112, 64, "swiglu")] + [("f32", *c) for c in [
        (1818, 128, 4160, "none"), (1601, 64, 4032, "gelu"),
        (74, 4416, 8640, "none"), (66, 3648, 6976, "silu"),
        (965, 128, 7360, "swiglu"), (1962, 64, 10112, "geglu"),
        (77, 1088, 6976, "swiglu"), (73, 2880, 4224, "geglu"),
        (65, 1280, 5440, "none"), (2437, 1408, 768, "silu"),
        (89, 1088, 3520, "swiglu"), (4951, 2432, 128, "geglu"),
        (375, 2048, 6848, "none")]]


@pytest.mark.parametrize("dtype,M,N,K,act",
                         [(t, *c) for c in LINEAR_GRAD
                          for t in ("bf16", "f32")] + LARGE_GRAD + FEW)
def test_linear_grad(dtype, M, N, K, act):
    half = ref.HALF[DT[dtype]]
    rounds = 1 if act == "none" else 2
    for bias, res in ((False, False), (True, True)):
        desc, t = linear_case(dtype, M, N, K, act, bias, res)
        names = [n for n in ("x", "w", "b", "w3", "b3")
                 if n in ("x", "w", "b") or act in ref.GATED]
        g = moe.LinearGrads(desc, device(), **{
            n: nan_like(t["x" if n == "x" else "w"].shape if n[0] != "b"
                        else (N,), DT[dtype]) for n in names})
        moe.moe_linear_grad(desc, t["x"], weights(t), t["dy"], g,
                            workspace(moe.moe_linear_grad_workspace_size(
                                desc)), dx_add=t["dx_add"])
        want = ref.linear_grad(act, half, *(f64(t[n]) for n in (
            "x", "w", "b", "w3", "b3", "dy", "dx_add")))
        for n in names:
            ref.check(getattr(g, n), want[n], half, rounds,
                      f"{n}, bias {bias}")


def dense_case(dtype, T, d, F, act, bias, seed=0):
    g, dt = generator(seed + T + 7 * d + 31 * F), DT[dtype]
    gated = act in ref.GATED
    t = {"x": normal(g, (T, d), 1.0, dt),
         "w1": normal(g, (F, d), d ** -0.5, dt),
         "w2": normal(g, (d, F), F ** -0.5, dt),
         "w3": normal(g, (F, d), d ** -0.5, dt) if gated else None}
    for n, size in (("b1", F), ("b2", d), ("b3", F)):
        t[n] = normal(g, (size,), 0.5, dt) \
            if bias and (gated or n != "b3") else None
    t["res"] = normal(g, (T, d), 1.0, dt) if bias else None
    t["dy"] = normal(g, (T, d), 1.0, dt)
    w = moe.DenseWeights(t["w1"], t["w2"], w3=t["w3"], b1=t["b1"],
                         b2=t["b2"], b3=t["b3"])
    return t, moe.DenseLayer(w, activation=act)


DENSE = [
    (1, 64, 64, "gelu"), (1, 1024, 2816, "swiglu"), (33, 320, 192, "silu"),
    (64, 64, 1024, "geglu"), (65, 128, 320, "swiglu"),
    (256, 64, 256, "gelu"), (1000, 1024, 704, "swiglu"),
    (2050, 2048, 1408, "swiglu"), (1537, 1088, 2048, "gelu"),
    (1057, 128, 8000, "silu"), (862, 192, 9920, "geglu"),
]
# (every product on its large tiles, the gradient of h among them)
DENSE_LARGE = [(2048, 1024, 4096, "silu"), (1500, 832, 7040, "swiglu"),
               (4100, 704, 2112, "geglu"), (2875, 384, 7296, "silu"),
               (6583, 448, 3136, "gelu")]
OF_BLOCK = ("x", "w1", "w2", "w3", "b1", "b2", "b3")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d,F,act", DENSE + DENSE_LARGE)
def test_dense(dtype, T, d, F, act):
    half = ref.HALF[DT[dtype]]
    for bias in (False, True):
        t, layer = dense_case(dtype, T, d, F, act, bias)
        args = [f64(t[n]) for n in OF_BLOCK]
        y = layer.forward(t["x"], residual=t["res"])
        # (h's rounding, then y's)
        ref.check(y, ref.dense(act, half, *args, f64(t["res"])), half, 2,
                  f"y, bias {bias}")
        g = layer.backward(t["x"], t["dy"], residual=bias).as_dict()
        want = ref.dense_grad(act, half, *args, f64(t["dy"]),
                              f64(t["dy"]) if bias else None)
        assert set(g) == {n for n in OF_BLOCK if t[n] is not None}
        for n in g:
            ref.check(g[n], want[n], half, 2, f"gradient of {n}, bias {bias}")
