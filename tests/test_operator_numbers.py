"""Numbers that do not fit the C ABI's int are refused on the host.  Nothing here reaches a kernel."""
import pytest
import torch

import speculative_decoding_verification_spec_gb300 as sv

from test_operator_refusals import host  # noqa: F401  (a fixture: no launch)
from test_round_devices import BF, I32, Reached, Ws, z


@pytest.mark.parametrize("far", [1 << 31, (1 << 32) + 16, 1 << 40, -(1 << 32) + 16])
def test_numbers_past_32_bits_are_refused(far, host):
    """The C ABI's int would keep their low bits: a window of 2^32 + 16 tokens would be one of 16."""
    ints = lambda *s: z(*s, dtype=I32)  # noqa: E731
    rows = z(3, 5, 2, 64, dtype=BF)
    cache = (z(4, 2, 16, 64, dtype=torch.uint8), z(4, 2, 16, 64, dtype=torch.uint8), z(4, 2), z(4, 2))
    pages = (ints(3, 2), ints(3), ints(3), ints(7), ints(1))
    out = dict(out=z(3, 5, 2, 64, dtype=BF), row_status=ints(3))

    def window(**kw):
        sv.verify_attention_window(rows, cache, ints(3, 2), ints(3), k=rows, v=rows, out=out, workspace=Ws(z(256, dtype=torch.uint8)), **kw)

    def reserve(**kw):
        sv.kv_pages_reserve(*pages, out=dict(slots=None, row_status=ints(3)), **kw)

    for f, kw in ((window, dict(window=far)), (window, dict(window=9, sinks=far)), (reserve, dict(page_size=far, max_new=5)),
                  (reserve, dict(page_size=16, max_new=far)), (lambda **kw: sv.kv_pages_release(*pages, out=dict(row_status=ints(3)), **kw),
                                                               dict(page_size=far))):
        with pytest.raises(ValueError):
            f(**kw)
    with pytest.raises(Reached):
        window(window=1 << 30, sinks=1 << 30)
