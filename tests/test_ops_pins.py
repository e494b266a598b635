"""Pins of the standalone operators' oracle (oracle/ops_ref.py) against torch in fp64 and closed forms.
No GPU needed."""

import numpy as np
import torch

from oracle import flint_moe_ref as R
from oracle import ops_ref as O


def test_q4_weight_reads_both_formats():
    # one byte per pair, low nibble first: codes 0..15 in order
    codes = np.array([[(2 * i) | ((2 * i + 1) << 4) for i in range(8)] * 8], dtype=np.uint8)      # [1][64] = 128 codes
    s = np.array([[0x3F00]], dtype=np.uint16)                                                        # bf16 0.5
    w = O.q4_weight("int4", codes, s)
    want = np.tile(np.array([0, 1, 2, 3, 4, 5, 6, 7, -8, -7, -6, -5, -4, -3, -2, -1]), 8) * 0.5
    np.testing.assert_array_equal(w[0], want)
    e4 = torch.tensor([1.0, 2.0, 0.5, 4.0, 8.0, 1.5, 0.25, 448.0]).to(torch.float8_e4m3fn).view(torch.uint8).numpy()[None]
    w = O.q4_weight("nvfp4", codes, e4, 2.0)
    grid = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0.0, -.5, -1, -1.5, -2, -3, -4, -6])
    want = np.concatenate([grid * v * 2.0 for v in (1.0, 2.0, 0.5, 4.0, 8.0, 1.5, 0.25, 448.0)])
    np.testing.assert_array_equal(w[0], want)


def test_q4_rotation_is_the_hadamard_of_both_sides():
    # rotated storage of W against rotated x is W x: store W Hn exactly (one code per row) and compare
    rng = np.random.default_rng(0)
    codes = rng.integers(0, 256, (5, 128), dtype=np.uint8)
    s = np.full((5, 2), 0x3F80, dtype=np.uint16)                                                     # 1.0
    x = rng.standard_normal((3, 256))
    w = O.q4_weight("int4", codes, s)
    unrotated = R.rotate_segments(w)                      # Hn is its own inverse
    np.testing.assert_allclose(O.q4_linear(x, "int4", codes, s, rotated=True), x @ unrotated.T, rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(O.q4_linear(x, "int4", codes, s), x @ w.T, rtol=1e-12, atol=1e-12)


def test_permute_is_a_stable_sort_with_dropped_ids():
    rng = np.random.default_rng(1)
    ids = rng.integers(-2, 9, (50, 3))
    off, perm, inv = O.expert_permute(ids, 7)
    flat = torch.from_numpy(ids.reshape(-1))
    key = torch.where((flat < 0) | (flat >= 7), torch.full_like(flat, 7), flat)
    order = torch.sort(key, stable=True).indices.numpy()
    kept = int((key < 7).sum())
    assert off[-1] == kept and np.array_equal(np.diff(off), np.bincount(key.numpy(), minlength=8)[:7])
    np.testing.assert_array_equal(perm[:kept], order[:kept])
    assert np.all(perm[kept:] == -1)
    flat_inv = inv.reshape(-1)
    assert np.array_equal(flat_inv >= 0, key.numpy() < 7)
    assert np.array_equal(perm[flat_inv[flat_inv >= 0]], np.nonzero(flat_inv >= 0)[0])


def test_grouped_and_combine_make_a_dense_mixture():
    # permute -> grouped -> combine equals the dense sum over experts with a routing matrix
    rng = np.random.default_rng(2)
    T, K, E, N, k = 6, 16, 4, 8, 2
    x, w = rng.standard_normal((T, K)), rng.standard_normal((E, N, K))
    ids = np.stack([rng.choice(E, k, replace=False) for _ in range(T)])
    ids[2, 1] = -1
    g = rng.random((T, k))
    off, perm, inv = O.expert_permute(ids, E)
    y, live = O.grouped_linear(x, w, off, rows=perm, row_div=k)
    assert live.sum() == T * k - 1
    got = O.expert_combine(y, inv, g, scale=0.5)
    dense = np.zeros((T, E))
    for t in range(T):
        for j in range(k):
            if ids[t, j] >= 0:
                dense[t, ids[t, j]] += g[t, j]
    np.testing.assert_allclose(got, 0.5 * np.einsum("te,enk,tk->tn", dense, w, x), rtol=1e-12, atol=1e-12)
    sw, _ = O.grouped_linear(x, w, off, rows=perm, row_div=k, swiglu=True)
    t = torch.from_numpy(y)
    np.testing.assert_allclose(sw, (torch.nn.functional.silu(t[:, :4]) * t[:, 4:]).numpy(), rtol=1e-12, atol=1e-12)


def test_grouped_ignores_offsets_outside_the_rows():
    x, w = np.ones((4, 8)), np.ones((3, 2, 8))
    y, live = O.grouped_linear(x, w, [-5, 2, 2, 99])
    assert live.all() and np.all(y == 8)
    _, live = O.grouped_linear(x, w, [0, 1, 1, 2])
    np.testing.assert_array_equal(live, [True, True, False, False])


def test_block_norm_closed_forms():
    rng = np.random.default_rng(3)
    x, y = rng.standard_normal((4, 32)), rng.standard_normal((4, 32))
    # without branch, scales and weights: the stack's rmsnorm
    x1, z = O.block_norm(x)
    np.testing.assert_array_equal(x1, x)
    np.testing.assert_allclose(z, R.rmsnorm(x, 1e-6), rtol=1e-12)
    # post-norm of a constant branch is 1 per element up to eps; a gate of +inf lets it through, -inf shuts it
    x1, _ = O.block_norm(x, np.full((4, 32), 3.0), post_norm=True, branch_scale=2.0, eps=1e-12)
    np.testing.assert_allclose(x1, x + 2.0, rtol=1e-9)
    x1, _ = O.block_norm(x, y, gate=np.full((1, 32), 800.0), sigmoid=True)
    np.testing.assert_allclose(x1, x + y, rtol=1e-12)
    x1, z = O.block_norm(x, y, gate=np.zeros((1, 32)), res_scale=0.5, pre_weight=np.full(32, 2.0))
    np.testing.assert_allclose(x1, 0.5 * x)
    t = torch.nn.functional.rms_norm(torch.from_numpy(0.5 * x), (32,), torch.full((32,), 2.0, dtype=torch.float64), 1e-6)
    np.testing.assert_allclose(z, t.numpy(), rtol=1e-12)
