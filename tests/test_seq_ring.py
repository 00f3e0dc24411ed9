"""The ring of work items in the packed and paged forward, checked in its
source on the host: a warp gives an item's place back only after a warp-wide
barrier, since lanes that have not yet read the item would read the next one."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "exact_attention_99_gb300", "csrc")


def test_every_release_of_an_item_follows_a_barrier_of_the_warp():
    text = open(os.path.join(CSRC, "fa_seq_fwd.cu")).read()
    arrivals = [m.start() for m in re.finditer(r"mbar_arrive\(&ctl\.it_empty", text)]
    assert arrivals
    for at in arrivals:
        before = [x.strip() for x in text[:at].rsplit("\n", 3)[1:]]
        assert "__syncwarp();" in before[:-1] and before[-1] == "if (lane == 0)", before
    # and all lanes of the warp come to it
    calls = re.findall(r"^(.*)\brelease\(i\);", text, flags=re.M)
    assert len(calls) == 4 and all("lane" not in c for c in calls), calls
