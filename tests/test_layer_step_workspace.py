"""Which workspaces a step's accumulated weights use: one of its number of rows, however many sequences come."""

from test_layer_mass_workspace import H_S, _decode, _layer, calls, layer  # noqa: F401


def test_a_steps_workspace_is_kept_and_large_enough(calls):  # noqa: F811
    lay = _layer()
    for n_seq in (1, 2, 5, 6, 7, 8, 100, 300, 9, 5, 1):
        _decode(lay, 5, n_seq)
        assert calls[-1][1].nbytes >= layer.attn_mass_workspace_size(5, H_S, n_seq)
    of = [w for _, w in calls]
    assert of[0] is of[1] is of[2] is of[-1] is of[-2]                   # no more sequences than rows: one
    assert of[3] is of[4] is of[5]                                       # few sizes beyond
    for n_seq in range(1, 1000):
        _decode(lay, 5, n_seq)
    assert len({w.data_ptr() for _, w in calls}) <= 9
    held = {w.data_ptr(): w for _, w in calls}
    _decode(lay, 5, 3)
    assert calls[-1][1].data_ptr() in held                               # (a recorded step may hold any of them)


def test_rows_of_their_own(calls):  # noqa: F811
    lay = _layer()
    _decode(lay, 5, 4)
    _decode(lay, 6, 4)
    assert calls[0][1].data_ptr() != calls[1][1].data_ptr()
