"""What happens when a bounded wait of the attention over the cache runs out, under the debug build's hook that leaves a
warp's first copy unissued: the call finishes, wcomp_device_check reports it, and the next calls are right."""
import pytest

pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_q4_moe_waits import COMMON, run  # noqa: E402

COPIES = COMMON + r"""
for name, B, n, H, share, D, rows in (("cluster", 1, 700, 2, 4, 128, 1), ("cut", 3, 4000, 4, 8, 128, 1), ("rows", 2, 900, 2, 5, 64, 3),
                                      ("256", 2, 3000, 2, 3, 256, 1)):
    width = -(-n // 64)
    c = W.kv4_create(B * width, H, D)
    table = torch.arange(B * width, dtype=torch.int32, device="cuda").view(B, width)
    lengths = torch.full((B,), n, dtype=torch.int32, device="cuda")
    W.kv4_append(c, draw(B * n, H, D), draw(B * n, H, D), table, lengths,
                 torch.arange(0, B * n + 1, n, dtype=torch.int32, device="cuda"))
    q = draw(B * rows, H * share, D)
    starts = torch.arange(0, B * rows + 1, rows, dtype=torch.int32, device="cuda")

    def call():
        lse, mass = torch.empty(B * rows, H * share, device="cuda"), torch.zeros(B, H, width * 64, device="cuda")
        return W.kv4_attend(c, q, table, lengths, starts, lse=lse, mass=mass), lse, mass

    want = call()
    run_out(1, call)
    assert L.wcomp_device_check(None) == W.ETIMEOUT, name
    assert L.wcomp_device_check(None) == W.OK, name
    assert all(torch.equal(x, y) for x, y in zip(call(), want)), name
    assert L.wcomp_device_check(None) == W.OK, name
    print("recovered", name)
"""


def test_copies_that_never_arrive():
    run(COPIES, "recovered", 4)
