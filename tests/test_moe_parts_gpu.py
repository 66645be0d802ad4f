"""The few-token layer where pieces are cut between pipelines and summed by the last of them to finish."""
from __future__ import annotations

import pytest
import torch

from test_moe_gpu import Layer, check, lib  # noqa: F401  (lib: the fixture)

pytestmark = pytest.mark.gpu

# tokens, experts, top k, H, I: on 152 SMs pieces are cut in the first product, the second, both, the second
CUT = [(1, 8, 2, 4224, 256), (1, 8, 2, 256, 2176), (1, 4, 2, 4224, 2176), (20, 6, 3, 2304, 1152)]


@pytest.mark.parametrize("T, E, k, H, I", CUT)
@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
def test_cut_pieces_give_the_same_bits_every_time(lib, T, E, k, H, I, fmt):  # noqa: F811
    # whichever pipeline comes last has to see what all others wrote: a part that it missed would change the sums
    p = Layer(T, E, k, H, I, fmt, seed=T + H, c=False)
    y = p.run(lib)
    check(y, *p.oracle())
    s = torch.cuda.Stream()
    ops = [torch.from_numpy(getattr(p, n)).cuda() for n in ("x", "sfx", "w13", "sf13", "w2", "sf2", "ids", "weights")]
    fn = lib.dg_moe_fp8_few_tokens if fmt == "e4m3" else lib.dg_moe_fp8_fp4_few_tokens
    many = torch.empty(300, T, H, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    for out in many:
        fn(*ops, None, out, stream=s)
    torch.cuda.synchronize()
    assert (many == y).all()
    assert lib.dg_get_device_status() == 0


@pytest.mark.parametrize("T, E, k, H, I", CUT)
@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
def test_waits_that_run_out_leave_the_counts_at_zero(lib, T, E, k, H, I, fmt):  # noqa: F811
    # every pipeline still counts its parts, in the second kernel only once the first has ended: the calls after it, before
    # the status is read (which clears the workspaces), are right
    p = Layer(T, E, k, H, I, fmt, seed=T + H + 1, c=False)
    y = p.run(lib)
    lib.dg_set_debug(1, 5_000_000)           # no weights are copied; waits give up after 5 ms
    try:
        p.run(lib)
    finally:
        lib.dg_set_debug(0, 0)
    for _ in range(3):
        assert torch.equal(p.run(lib), y)
    assert lib.dg_get_device_status() == 5   # DG_ERR_TIMEOUT, from the second call
    assert torch.equal(p.run(lib), y) and lib.dg_get_device_status() == 0
