"""Row strides given to qlinear_bf16: the tensors have to reach the last row."""
import pytest

from tests._call_cpu import calls

torch = pytest.importorskip("torch")

BF = torch.bfloat16
M, N, K = 3, 32, 64


def _args(x=None, y=None, ldx=None, ldy=None, M=M, out=0):
    x = torch.zeros((M, K), dtype=BF) if x is None else x
    y = torch.zeros((M, N), dtype=torch.float32 if out else BF) if y is None else y
    w = [torch.zeros((N, n), dtype=torch.uint8) for n in (K // 2, K // 16)]
    return [x, *w, torch.ones(1), y, M, N, K, None, out, 0, ldx, ldy, 0]


def test_strides_that_fit():
    c = calls()
    wide = torch.zeros((M, 200), dtype=BF)
    for x, ldx in ((torch.zeros((M, K), dtype=BF), K), (wide, 200), (wide[:, :K], 200), (wide[:, 136:], 200),
                   (wide[0], 200), (torch.zeros(2 * 72 + K, dtype=BF), 72), (wide[:, :K], 104)):
        a = c.ok("qlinear_bf16", *_args(x=x, ldx=ldx))
        assert a[0] == x.data_ptr() and a[1] == ldx
    for y, ldy in ((torch.zeros((M, N), dtype=BF), N), (torch.zeros((M, 40), dtype=BF)[:, 8:], 40),
                   (torch.zeros(2 * 33 + N, dtype=BF), 33)):
        a = c.ok("qlinear_bf16", *_args(y=y, ldy=ldy))
        assert a[9] == y.data_ptr() and a[10] == ldy
    # one row needs its width, whatever the stride
    c.ok("qlinear_bf16", *_args(x=torch.zeros(K, dtype=BF), y=torch.zeros(N, dtype=BF), ldx=1 << 20, ldy=1 << 62, M=1))
    c.ok("qlinear_bf16", *_args(y=torch.zeros(2 * 33 + N), ldy=33, out=1))


def test_strides_past_the_tensors_end_are_refused():
    c = calls()
    wide = torch.zeros((M, 200), dtype=BF)
    for x, ldx in ((torch.zeros((M, K), dtype=BF), K + 8), (torch.zeros((M - 1, K), dtype=BF), K), (wide[:, 144:], 200),
                   (wide[1], 200), (torch.zeros(2 * 72 + K - 1, dtype=BF), 72), (wide, 1 << 31), (wide, 1 << 62)):
        c.refused("qlinear_bf16", *_args(x=x, ldx=ldx), match="x: ")
    for y, ldy in ((torch.zeros((M, N), dtype=BF), N + 1), (torch.zeros((M - 1, N), dtype=BF), N),
                   (torch.zeros(2 * 33 + N - 1, dtype=BF), 33), (torch.zeros((M, N), dtype=BF), 1 << 62),
                   (torch.zeros((M, N), dtype=BF), (1 << 63) - 1)):
        c.refused("qlinear_bf16", *_args(y=y, ldy=ldy), match="y: ")
    c.refused("qlinear_bf16", *_args(y=torch.zeros(2 * 33 + N - 1), ldy=33, out=1), match="y: ")
    c.refused("qlinear_bf16", *_args(x=torch.zeros(K - 1, dtype=BF), ldx=K, M=1), match="x: ")
