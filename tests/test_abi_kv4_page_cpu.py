"""Page sizes that the cache calls refuse, whatever their size: the refusal
returns (a call that does not is ended with its process)."""
import subprocess
import sys

import pytest

PAGES = [-1, -2 ** 31, 0, 1, 8, 15, 17, 2048, 1 << 30, (1 << 30) + 1, (1 << 31) - 1]

CALL = """
import mixed_precision_quantized_act_amd as qa
from tests.test_abi_attn_cpu import P, _kv
fn, page = {fn!r}, {page}
if fn == "attn_kv4":
    args = dict(q=P(0), ldq=256, B=2, Lq=1, Hq=4, H=2, D=64, k_q=P(2), k_s=P(3), v_q=P(4), v_s=P(5), k_ts=P(6),
                v_ts=P(7), pages=8, page=page, table=P(8), max_pages=4, lens=P(9), q_lens=None, causal=1, scale=0.125,
                o=P(10), ldo=256, ws=None, ws_bytes=0, stream=None)
else:
    args = {{**_kv(T=1), "page": page}}
assert getattr(qa.lib(), fn)(*args.values()) == -2       # QA_ESHAPE
"""


@pytest.mark.parametrize("fn", ["kv4_append", "kv4_read", "attn_kv4"])
def test_every_bad_page_is_refused(fn):
    # one process for all sizes: it returns within seconds or not at all
    code = "\n".join(CALL.format(fn=fn, page=p) for p in PAGES)
    subprocess.run([sys.executable, "-c", code], check=True, timeout=100)
