"""Which forms of the output head's losses the GPU tests' sizes take, read off the workspace's parts; and that the bound
of f32 gradients tells g in three parts of bf16 from g in two."""
import pytest
import torch

from head_forms import BATCH, FORMS, PIECES, STREAMED, THREE_PARTS


@pytest.fixture(scope="module")
def size():
    import block_scaled_precision_bsq_amd as b
    return b.bsq_linear_loss_workspace_size


def up(n, m):
    return -(-n // m) * m


def tile(size, T, V, H):
    """Columns of a tile of logits: lists of one entry add four numbers a token, and the table of its tiles."""
    table = size(T, H, V, 1) - size(T, H, V, 0) - 4 * up(4 * T, 256)
    return [n for n in (64, 128, 256) if up(2 * T * (-(-V // n) + 1), 256) == table]


@pytest.mark.parametrize("name", [*FORMS, *STREAMED])
def test_forms(size, name):
    T, V, H, block, on_x = (FORMS | STREAMED)[name]
    assert block in tile(size, T, V, H)
    # dw of a copy reads its transpose
    assert (size(T, H, V, 0, 3) == size(T, H, V, 0, 1)) == on_x
    assert (name in STREAMED) == (2 * V * H > 1 << 28)


def test_pieces(size):
    T, V, H, columns = PIECES
    Tp, Hp = up(T, 256), up(H, 64)
    g = size(T, H, V, 0, 2, 1) - 256 - 2 * up(4 * Tp, 256) - 2 * up(2 * Tp * Hp, 256)
    assert g == 2 * 3 * Tp * columns and columns < V


def test_batches(size):
    T, V, blocks = BATCH
    for rows, block in blocks.items():
        assert tile(size, rows, V, 136) == [block]


def test_three_parts():
    """The bound lies between the two: g in parts of bf16, of values spread over a few binades."""
    g = torch.Generator().manual_seed(0)
    v = torch.exp(torch.randn(1 << 16, generator=g)) / 33000
    errors, rest = [], v.double()
    for _ in range(3):
        rest = rest - rest.float().bfloat16().double()
        errors.append((rest.norm() / v.double().norm()).item())
    assert errors[1] > 1.25 * THREE_PARTS and errors[2] < THREE_PARTS / 50
