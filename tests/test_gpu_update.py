"""The orthogonalised update against the polynomial in 64 bits where its accuracy can go wrong: few and many steps,
gradients of a few strong directions."""
import pytest
import torch

import gemms_linear_layers_gb300 as tg
from gemms_linear_layers_gb300 import inputs
import block_ref as R

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
QUINTIC = (3.4445, -4.7750, 2.0315)


def randn(shape, tag):
    return inputs.normal(shape, 1.0, F32, inputs.seed_for("update", *shape, tag)).cuda()


def gradient(batch, rows, cols, noise, dtype=F32, rank=8):
    """A strong part of this rank, its directions of sizes 1 to 0.1, beside `noise`."""
    left = randn((batch, rows, rank), "left") * 0.7 ** torch.arange(rank, device="cuda")
    return (left @ randn((batch, rank, cols), "right") + noise * randn((batch, rows, cols), "noise")).to(dtype)


def polynomial(G, coeffs, scale=1.0, eps=1e-7):
    """The definition in 64 bits, of a batch."""
    X = G.double()
    X = X / (torch.linalg.vector_norm(X, dim=(1, 2), keepdim=True) + eps)
    tall = X.shape[1] > X.shape[2]
    X = X.mT if tall else X
    for a, b, c in coeffs:
        A = X @ X.mT
        X = a * X + (b * A + c * (A @ A)) @ X
    return scale * (X.mT if tall else X)


def errors(got, ref):
    """Of each matrix, in the Frobenius norm: the result's error, and that of rounding the true values once."""
    size = lambda t: torch.linalg.vector_norm(t, dim=(1, 2))  # noqa: E731
    return size(got.double() - ref) / size(ref), size(ref.to(got.dtype).double() - ref) / size(ref)


# What the parts leave is independent of the result's rounding, so that squares add.  A step leaves at most 2^-17 of
# |X| in X (0.71 of that and less in the mean square), which later steps enlarge by at most a each: 57 times in
# four steps of a = 3.4445, 3.1e-4 beside |O| of at least 0.7 sqrt(8) = 2.  Rounding to bf16 is 1.66e-3 in the mean
# square: 1.5e-4 adds 0.4 % to it, and 2 % is a fifth of it.
@pytest.mark.parametrize("noise", (0.3, 0.02, 1e-3))
@pytest.mark.parametrize("steps", (2, 3, 4))
@pytest.mark.parametrize("rows,cols", [(300, 700), (577, 321)])
def test_a_bf16_result_of_few_steps_has_its_rounding_alone(rows, cols, steps, noise):
    G = gradient(2, rows, cols, noise)
    off, rounding = errors(tg.tg_orthogonalize(G, steps=steps), polynomial(G, [QUINTIC] * steps))
    assert bool((off <= 1.02 * rounding).all()), (off / rounding).tolist()


# Steps of a = 3.4445 enlarge what a step leaves in X by 198 in all over five, 683 over six, beside |O| of at least 2.
# Values are stored to 2^-22, three of them in a step, and summed in FP32: at these sizes what a step leaves is held to
# 2^-20 of |X|.
def left(steps):
    return sum(3.4445 ** i for i in range(steps)) / 2 * 2.0 ** -20


@pytest.mark.parametrize("out", (BF, HF))
@pytest.mark.parametrize("noise", (0.02, 1e-3, 1e-4))
@pytest.mark.parametrize("steps", (5, 6))
@pytest.mark.parametrize("rows,cols", [(300, 700), (577, 321)])
def test_weak_directions_keep_their_digits(rows, cols, steps, noise, out):
    G = gradient(2, rows, cols, noise)
    off, rounding = errors(tg.tg_orthogonalize(G, steps=steps, out_dtype=out), polynomial(G, [QUINTIC] * steps))
    assert bool((off <= torch.hypot(rounding, torch.full_like(off, left(steps)))).all()), (off.tolist(), rounding.tolist())


@pytest.mark.parametrize("steps", (1, 5))
def test_each_matrix_has_its_own_size_beside_eps(steps):
    """Gradients far below eps, of eps' size and far above it in one batch: X's norm runs from 1e-20 to 1."""
    sizes = torch.tensor([1.0, 1e-27, 1e3, 1e-8, 3e-10, 1e-12, 0.0, 1e-18], device="cuda")
    G = gradient(8, 130, 200, 0.02) * sizes[:, None, None]
    got = tg.tg_orthogonalize(G, steps=steps)
    live = sizes > 0
    off, rounding = errors(got[live], polynomial(G[live], [QUINTIC] * steps))
    # not by hypot: with what is left far below the rounding, the two's product over the 26,000 entries of a matrix
    # (2 x 1.7e-3 x 1e-6 / sqrt(26,000) = 2e-11) outweighs its square (1e-12)
    assert bool((off <= 1.02 * rounding).all()), (off / rounding).tolist()
    assert not got[6].any()
    for i in range(8):
        assert torch.equal(got[i], tg.tg_orthogonalize(G[i], steps=steps))


# Coefficients whose polynomial has a zero, or lets X grow: two bf16 parts.
@pytest.mark.parametrize("coeffs", (((2.0, -3.0, 1.0), (3.0, -3.5, 1.25)), ((8.0, 30.0, 20.0), (8.0, 30.0, 20.0)),
                                    ((0.0, 1.0, 0.5),), ((0.0, 0.0, 2.0), (1.0, 0.0, 0.0))))
def test_sizes_that_coefficients_do_not_bound(coeffs):
    G = gradient(2, 150, 90, 0.3)
    got = tg.tg_orthogonalize(G, coeffs=coeffs, out_dtype=BF)
    assert "bf16 parts" in tg.tg_last_call()
    for g, o in zip(G, got):
        ref, noise = R.orthogonalize(g, coeffs, 1.0, 1e-7, HF)  # two parts, 2^-17
        size = torch.linalg.vector_norm(ref)
        assert torch.linalg.vector_norm(o.double() - ref) <= noise + 2.0 ** -8 * size


def check(got, ref, leftover, what):
    """Each matrix against its true values: in the Frobenius norm as above, and every element within half a step of its
    own and 2^-8 of the matrix's root mean square (a normal variable stays within 12 times its deviation, and
    `leftover`, what the parts and sums leave of a result's size, is at most 3e-4 in these tests: 12 x 3e-4 < 2^-8)."""
    off, rounding = errors(got, ref)
    assert bool((off <= rounding + leftover).all()), (what, off.tolist(), rounding.tolist())
    half = R.half_step(torch.maximum(got.double().abs(), ref.abs()), got.dtype)
    rms = ref.square().mean((1, 2), keepdim=True).sqrt()
    assert bool(((got.double() - ref).abs() <= half + 2.0 ** -8 * rms).all()), what


# The kernel's instances (tiles of up to 128 columns or wider, tall or not) at each width that the rule takes on 152
# SMs, with and without a strip of a last row tile (a smaller side of a multiple of 256 and at most 128 more), and sizes
# off the tiles and off 8.  A changed rule has to choose its own sizes here.
@pytest.mark.parametrize("batch,rows,cols,width", [
    (1, 130, 200, 64), (1, 200, 130, 64), (1, 313, 331, 64), (1, 331, 313, 64), (3, 137, 333, 64),
    (24, 252, 264, 128), (24, 264, 252, 128), (1, 374, 398, 128), (1, 398, 374, 128), (2, 1301, 1999, 128),
    (17, 700, 700, 128), (1, 1700, 2900, 128), (1, 2901, 1699, 128),
    (40, 130, 137, 192), (40, 191, 130, 192), (1, 2304, 2304, 192), (30, 500, 900, 192), (29, 903, 501, 192),
    (40, 252, 398, 256), (39, 397, 255, 256), (40, 313, 398, 256), (40, 801, 264, 256), (24, 576, 576, 256),
    (20, 1100, 513, 256), (3, 1500, 1500, 256), (6, 1401, 1003, 256), (2, 1799, 1801, 256), (16, 449, 448, 256)])
def test_every_width_of_tiles(batch, rows, cols, width):
    G = gradient(batch, rows, cols, 0.02)
    got = tg.tg_orthogonalize(G, steps=3)
    assert f"tiles=256x{width} fp16 parts" in tg.tg_last_call(), tg.tg_last_call()
    check(got, polynomial(G, [QUINTIC] * 3), 1e-4, (batch, rows, cols))
    # the same call gives the same bits.  A matrix alone may not: its tiles may have another width, and tiles of 192
    # columns take other elements of the symmetric matrices from across the diagonal, where the two cross products
    # were added in the other order
    assert torch.equal(tg.tg_orthogonalize(G, steps=3), got)


def test_the_large_tall_batch():
    G = gradient(4, 5760, 2304, 0.02, BF)
    got = tg.tg_orthogonalize(G, steps=2)
    assert "tiles=256x256 fp16 parts" in tg.tg_last_call()
    check(got, polynomial(G, [QUINTIC] * 2), 1e-4, "4 x 5,760 x 2,304")


CUBIC = ((2.0, -1.5, 0.5), (1.875, -1.25, 0.375), (1.5, -0.5, 0.0))
VARIED = ((4.0, -6.0, 2.8), (3.2, -3.0, 1.0), (2.5, -2.0, 0.6), (2.0, -1.5, 0.5), (1.875, -1.25, 0.375), (1.5, -0.5, 0.0))


@pytest.mark.parametrize("out", (BF, HF))
@pytest.mark.parametrize("coeffs", (CUBIC, VARIED[:2], VARIED[:4], VARIED, VARIED[::-1], (QUINTIC,) * 2 + CUBIC))
def test_a_triple_for_each_step(coeffs, out):
    for rows, cols in ((70, 130), (200, 90)):
        G = gradient(2, rows, cols, 0.1)
        got = tg.tg_orthogonalize(G, coeffs=coeffs, scale=0.5, out_dtype=out)
        assert "fp16 parts" in tg.tg_last_call()
        # no step here has a above 4, and a gradient of noise 0.1 has few directions below 1e-2 of its strongest
        check(got, polynomial(G, coeffs, 0.5), 1e-4, (rows, cols))
        assert torch.equal(got, tg.tg_orthogonalize(G, coeffs=[list(k) for k in coeffs], steps=len(coeffs), scale=0.5, out_dtype=out))


@pytest.mark.parametrize("out", (BF, HF))
@pytest.mark.parametrize("steps", (1, 2, 3, 4, 5, 6, 9))
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 9), (31, 33), (257, 256)])
def test_numbers_of_steps(rows, cols, steps, out):
    G = gradient(2, rows, cols, 0.3)
    check(tg.tg_orthogonalize(G, steps=steps, out_dtype=out), polynomial(G, [QUINTIC] * steps), 1e-4, (rows, cols, steps))


@pytest.mark.parametrize("steps", (1, 5))
@pytest.mark.parametrize("size,eps,scale", [(1.0, 1e-7, 1e38), (1.0, 1e-7, 1e-36), (1e-30, 1.0, 1.0), (1e-33, 1.0, 1.0), (1e-33, 1.0, -1e30),
                                            (1e30, 1e-7, 3e37), (0.0, 1.0, 3e38)])
def test_results_near_the_ends_of_the_range(size, eps, scale, steps):
    """Of the gradient, of X beside a large eps, and of the result, which is a normal bf16 number here."""
    G = gradient(2, 60, 90, 0.1) * size
    got = tg.tg_orthogonalize(G, steps=steps, scale=scale, eps=eps)
    ref = polynomial(G, [QUINTIC] * steps, scale, eps)
    if size == 0.0:
        assert not got.any()
        return
    assert bool(got.isfinite().all())
    by = 1.0 / ref.abs().amax()  # the same in the middle of the range: half steps of the smallest results aside
    off = torch.linalg.vector_norm((got.double() - ref) * by)
    assert off <= (2.0 ** -8 + 1e-4) * torch.linalg.vector_norm(ref * by), float(off)


@pytest.mark.parametrize("out", (BF, F32))
@pytest.mark.parametrize("coeffs", (((100.0, 0.0, 0.0),) * 4, ((30.0, 5.0, 2.0), (2.0, 1e-4, 1e-9)), ((1e-3, 0.0, 0.0),) * 3,
                                    ((-0.02, -0.01, -0.001), (-5.0, 100.0, 1e5), (1.5, -0.5, 0.1)), ((1e8, 1e7, 1e6),)))
def test_growth_and_decay_that_coefficients_bound(coeffs, out):
    if out == F32:  # of G, with a result in fp16's range
        top = 1.0
        for a, b, c in coeffs:
            top = abs(a * top + b * top ** 3 + c * top ** 5)
        G, scale, out = gradient(2, 90, 140, 0.1), 1.0 / top, HF
    else:
        G, scale = gradient(2, 90, 140, 0.1, BF), 1.0
    got = tg.tg_orthogonalize(G, coeffs=coeffs, scale=scale, out_dtype=out)
    assert "fp16 parts" in tg.tg_last_call(), tg.tg_last_call()
    ref = polynomial(G, coeffs, scale)
    off = torch.linalg.vector_norm(got.double() - ref, dim=(1, 2)) / torch.linalg.vector_norm(ref, dim=(1, 2))
    assert bool((off <= torch.finfo(out).eps / 2 + 1e-4).all()), off.tolist()
