"""The bounded waits of the attention kernels running out (needs a B200).

tria_set_attention_wait_limit(1) makes the first wait that is not already
satisfied run out: the kernel must set status bit 1, let its own loads and MMAs
land, free its tensor memory and return.  Every barrier still completes; the
waits are cut short from inside the kernel, and nothing faults.  An ordinary
call afterwards must be right (tensor memory left allocated, or a copy in
flight, would break it).
"""
from __future__ import annotations

import time

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import key_retention_scoring_b200 as T  # noqa: E402
from key_retention_scoring_b200 import build as tria_build  # noqa: E402
from tests.serving_helpers import Store  # noqa: E402
from tests.test_gpu_prompt_attention import Prompt  # noqa: E402
from tests.test_gpu_tree_attention import Drafts  # noqa: E402

WAIT_EXPIRED = 2


@pytest.fixture(scope="module", autouse=True)
def _built():
    tria_build.build()
    yield
    torch.cuda.empty_cache()


def expire(call, ws):
    """The call under a limit of 1 ns: ends at once.  Whether a wait ran out."""
    T.tria_read_device_status(ws)
    T.tria_set_attention_wait_limit(1)
    try:
        t0 = time.monotonic()
        call()
        flags = T.tria_read_device_status(ws)  # synchronises the stream
        # loads of a few us are waited for; a load looked for in the wrong phase of
        # its barrier would be waited for until the drain's own 2 s are over
        assert time.monotonic() - t0 < 1.9
    finally:
        T.tria_set_attention_wait_limit(0)
    assert flags in (0, WAIT_EXPIRED), flags
    assert T.tria_read_device_status(ws) == 0
    return flags != 0


# one block with all its loads issued before any wait; several items for a
# processor; more blocks than a ring has stages
@pytest.mark.parametrize("lens", [[5], [300, 40, 1], [4000, 900], [1 + (37 * i) % 190 for i in range(120)]],
                         ids=["one", "short", "long", "many"])
def test_prompt_wait_expires_and_the_next_call_is_right(lens):
    p = Prompt(32, 8, lens, seed=21, lead=3, tail=5)
    expired = 0
    for _ in range(3):
        p.out.fill_(7.0)
        p.lse.fill_(7.0)
        if expire(p.run, p.ws):
            expired += 1
        else:
            # the limit is looked at when a sleep has run out, and all waits may have
            # ended within theirs (one short item's do): then the call is an ordinary one
            p.check(seqs=range(0, len(lens), 17), heads=[0, 31])
        p.untouched()
    assert expired or lens == [5]
    p.run()
    p.check(seqs=range(0, len(lens), 17), heads=[0, 31])
    assert T.tria_read_device_status(p.ws) == 0


# up to 128 rows for a KV head, and more; one line of key blocks, and one for each head
@pytest.mark.parametrize("block", [0, 16])
@pytest.mark.parametrize("n_draft", [9, 40])
def test_tree_wait_expires_and_writes_no_rows_of_other_calls(block, n_draft):
    st = Store(T, 1, 32, 8, [20011, 37, 9000], 20064, block=block, seed=22)
    try:
        d = Drafts(st, 32, [n_draft, 3, n_draft], seed=22)
        n = d.out.shape[0]
        far = Drafts(st, 32, [50, 52, 60], seed=23)        # its shared units' rows lie behind n
        ws = T.alloc_workspace(max(d.ws.numel(), far.ws.numel()))
        far.ws = d.ws = ws
        out = torch.full((256, 32, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((256, 32), 7.0, device="cuda")
        d.out, d.lse = out[16: 16 + n], lse[16: 16 + n]
        g = torch.Generator(device="cuda").manual_seed(24)
        for held in ("another call's records", "anything"):
            expired = 0
            for _ in range(3):
                far.run()
                if held == "anything":
                    ws.copy_(torch.randint(0, 256, ws.shape, generator=g, device="cuda", dtype=torch.uint8))
                expired += expire(d.run, ws)
                for x in (out, lse):
                    assert bool((x[:16] == 7.0).all()) and bool((x[16 + n:] == 7.0).all()), held
            assert expired, held
        d.run()
        d.check(heads=[0, 13, 31])
        assert T.tria_read_device_status(ws) == 0
    finally:
        st.free()
