"""Feed-forward calls that reach every launch the library has for them: (path, kind, dtype, act, bias,
residual, kept sums, M, N, K).  The paths are those of ffn_path_query.cu; test_ffn_paths_host.py checks
that the calls take them."""
DTYPES = ("f32", "bf16", "f16")
ACTS = ("none", "relu", "relu2", "silu", "gelu", "gelu_tanh")


def _linear(dt, act, bias, residual, keep, shapes, odd):
    """Shapes are (path, tokens, row tiles, chunks).  Rows of 16-byte multiples (outputs leave by TMA) and
    odd ones (element by element); the last chunk is never full."""
    return [(path, "linear", dt, act, bias, residual, keep, M, 128 * tn - d, 128 * kc - 32)
            for path, M, tn, kc in shapes for d in (8, odd)]


def _gated(dt, act, bias, keep, shapes):
    return [(path, "gated", dt, act, bias, False, keep, M, 64 * tn - d, 128 * kc - 32)
            for path, M, tn, kc in shapes for d in (8, 1)]


FORWARD = (
    _linear("bf16", "silu", True, True, False, [
        ("16/1/c2", 400, 1, 24), ("16/1/c4", 3, 1, 24), ("16/1/leftover", 3, 152, 32), ("16/1/splitS", 3, 1, 80),
        ("32/1/c2", 1100, 1, 40), ("32/1/c4", 600, 1, 80), ("32/1/leftover", 17, 152, 48), ("32/1/splitS", 400, 1, 160),
        ("64/1/leftover", 1537, 6, 112), ("64/1/splitS", 1200, 1, 160), ("64/1/whole+", 1200, 15, 32),
        ("128/1/leftover", 200, 75, 80), ("128/1/splitS", 1537, 2, 240), ("128/1/whole", 2500, 4, 24),
        ("128/1/whole+", 2000, 14, 48), ("192/1/leftover", 1537, 17, 112), ("192/1/splitS", 2100, 3, 240),
        ("192/1/whole", 2100, 9, 24), ("192/1/whole+", 1700, 32, 24)], 3) +
    _linear("f32", "gelu", True, True, True, [
        ("16/1/c4", 3, 1, 24), ("32/1/c2", 1100, 1, 48), ("32/1/leftover", 800, 6, 160), ("64/1/splitS", 1200, 1, 240),
        ("128/1/leftover", 1537, 17, 112), ("128/1/whole+", 2000, 14, 64), ("128/2/whole+", 2500, 124, 1),
        ("192/1/leftover", 2100, 18, 112), ("192/1/whole+", 1700, 32, 32)], 1) +
    _linear("f16", "none", False, False, False, [
        ("32/1/c4", 600, 1, 64), ("64/1/leftover", 1537, 6, 160), ("128/1/splitS", 1537, 2, 160),
        ("192/1/splitS", 2100, 3, 240), ("192/1/whole", 2100, 9, 12)], 5) +
    _gated("bf16", "silu", False, False, [
        ("16/1/c2", 400, 1, 24), ("16/1/c4", 3, 1, 24), ("16/1/leftover", 3, 152, 32), ("32/1/c4", 600, 1, 64),
        ("64/1/leftover", 1537, 6, 160), ("64/1/splitS", 1200, 1, 160), ("64/1/whole+", 1200, 15, 17), ("128/1/leftover", 200, 75, 64), ("128/1/whole+", 2000, 14, 32),
        ("192/1/leftover", 1537, 17, 112), ("192/1/splitS", 2100, 3, 240), ("192/1/whole", 2100, 9, 12),
        ("192/1/whole+", 2500, 15, 24)]) +
    _gated("f32", "silu", True, True, [
        ("32/1/c2", 800, 1, 40), ("32/1/splitS", 400, 1, 160), ("128/1/leftover", 200, 75, 80),
        ("128/1/whole+", 2000, 14, 40), ("192/1/splitS", 2100, 3, 240)]) +
    _gated("f16", "gelu", True, True, [
        ("16/1/splitS", 3, 1, 80), ("32/1/leftover", 17, 152, 48), ("128/1/splitS", 1537, 2, 240),
        ("192/1/leftover", 1537, 17, 112), ("192/1/whole+", 1700, 32, 17)]) +
    # several rows per thread: from 64 and from 128 rows per SM on
    [("decode/2", "linear", "bf16", "relu", True, True, True, 1, 9473, 4064),
     ("decode/2", "gated", "f16", "silu", True, False, False, 1, 5001, 4096),
     ("decode/4", "linear", "f32", "gelu", True, True, True, 1, 19001, 8160),
     ("decode/4", "gated", "bf16", "silu", True, False, True, 1, 14336, 4096),
     ("decode/4", "gated", "f32", "gelu_tanh", False, False, False, 1, 14337, 4064),
     ("decode/2", "linear", "f16", "silu", True, True, False, 2, 9473, 4064),
     ("decode/4", "gated", "bf16", "gelu", True, False, True, 2, 14337, 4096)]
)


def _gradient(kind, dt, act, shapes):
    """Shapes are (path, tokens, column tiles of dx, chunks of weight rows)."""
    gated = kind == "gated_grad"
    return [(path, kind, dt, act, True, False, False, M, (64 if gated else 128) * rc - 3, 128 * kt - 32)
            for path, M, kt, rc in shapes]


GRADIENT = (
    _gradient("linear_grad", "f32", "gelu_tanh", [
        ("16/1/c2", 100, 1, 24), ("16/1/leftover", 3, 152, 40), ("16/1/splitS", 3, 1, 80), ("32/1/c2", 200, 1, 32),
        ("32/1/leftover", 5, 152, 48), ("64/1/splitS", 260, 1, 160), ("128/1/leftover", 150, 38, 80),
        ("128/1/splitS", 800, 1, 160), ("192/1/leftover", 1400, 5, 112), ("192/1/splitS", 1700, 1, 240),
        ("192/1/whole+", 2500, 4, 12), ("192/2/whole+", 2500, 4, 1)]) +
    _gradient("linear_grad", "bf16", "gelu", [
        ("16/1/c2", 129, 1, 24), ("16/1/leftover", 3, 152, 40), ("32/1/c4", 129, 1, 48), ("32/1/splitS", 80, 1, 160),
        ("64/1/leftover", 1537, 2, 160), ("64/1/whole+", 333, 17, 1), ("128/1/splitS", 1000, 1, 160),
        ("192/1/leftover", 1100, 8, 112), ("192/1/splitS", 2000, 1, 240), ("192/1/whole+", 2000, 6, 12),
        ("192/2/whole+", 2000, 6, 1)]) +
    _gradient("gated_grad", "bf16", "silu", [
        ("16/1/c4", 3, 1, 24), ("32/1/c2", 260, 1, 32), ("32/1/leftover", 9, 152, 48), ("64/1/splitS", 700, 1, 80),
        ("128/1/leftover", 200, 38, 80), ("128/1/whole+", 1537, 6, 1), ("192/1/leftover", 1100, 8, 112),
        ("192/1/whole", 2000, 3, 1)]) +
    _gradient("gated_grad", "f16", "relu2", [
        ("16/1/splitS", 3, 1, 80), ("64/1/leftover", 1537, 2, 160), ("192/1/splitS", 2000, 1, 240)])
)

# More than 1024 tokens and 2304 rows: the digits, then column sums by blocks of four warps in clusters of
# four to eight, then the product.  (M, N of a linear layer, K); gated: N / 2.
COLUMNS = ((1025, 2502, 96), (1100, 4000, 64), (1027, 14340, 32), (1030, 33002, 32), (2048, 2434, 32))
