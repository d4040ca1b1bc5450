"""A batch of no sequences, whose table and lengths have no memory, on the host:
every call returns before any CUDA call."""
import exact_tiled_attention_23_gb300 as fa
from test_paged_abi import append, cache, fwd


def test_no_sequences_need_no_table():
    fa.build()
    none = dict(table=None, seq_len=None)
    assert fwd(cache(**none), B=0, prefix=None) == fa.FA_OK
    assert fwd(cache(**none), B=0, prefix=7) == fa.FA_OK
    assert append(cache(**none), B=0) == fa.FA_OK
    assert fa.fa_fwd_paged_workspace_bytes(cache(**none), 0, 4, 1) == 0
    # one sequence does
    for part in ("table", "seq_len"):
        assert fwd(cache(**{part: None}), B=1, prefix=None) == fa.FA_ERR_INVALID_ARG
        assert append(cache(**{part: None}), B=1) == fa.FA_ERR_INVALID_ARG
