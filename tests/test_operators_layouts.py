"""Layouts that the population operators take, told by what a call is refused for: no GPU is needed, and the pointers
handed over are never followed."""
from test_operators_host import FAKE, _prompt, _scan, lib  # noqa: F401


def test_scan_takes_states_at_any_element(lib):
    """A layer's part of a larger cache starts wherever the sizes put it. The workspace is what is refused here."""
    for io, cfg, status in ((dict(conv_in=FAKE + 2, conv_out=FAKE + 6), {}, 3), (dict(conv_in=FAKE + 1), {}, 1), (dict(conv_out=FAKE + 2), dict(dtype=0), 1),
                            (dict(ssm_in=FAKE + 4, ssm_out=FAKE + 12, xbc_stride=1000), dict(state_dim=63), 3),
                            (dict(ssm_in=FAKE + 2, xbc_stride=1000), dict(state_dim=63), 1), (dict(ssm_out=FAKE + 4), {}, 1)):
        c, w, i = _scan(io, **cfg)
        assert _prompt(lib, c, w, i, None, 0) == status, (io, cfg)
