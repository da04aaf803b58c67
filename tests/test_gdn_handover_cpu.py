"""The hand-over between the warps of the per-head prefill's state kernel, as a
model on the host: whatever wait runs out, at whatever place, every warp comes
to the end of its loop, so that the CTA can report it and leave.

The warps' programs are read from the kernel's source: the order in which a role
arrives at and waits for the named barriers, waits for mbarriers and commits
products.  A named barrier counts arrivals, whoever they come from; a warp that
arrives twice within one phase takes another's place there."""
import os
import random
import re

import pytest

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                   "linear_attention_serving_gated_gb300", "csrc", "gdn_prefill.cu")
CHAIN = 3  # chain warps of the model
OPS = re.compile(r"(?P<arrive>(?:chain|barrier)_arrive<[^>]*>\((?P<a_id>kBar\w+)(?P<held>, ok)?\))"
                 r"|(?P<sync>chain_await<[^>]*>\((?P<s_id>kBar\w+)\))"
                 r"|(?P<wait>(?:chain|warp)_wait\(&bars\.(?P<w_id>\w+)(?:\[\w+\])?, (?P<phase>[^;]*?)\)[;)])"
                 r"|(?P<commit>mma_commit\(&bars\.(?P<c_id>\w+))"
                 r"|(?P<past>(?P<later>if \(c > 0\) )?past_(?P<p_kind>arrive|await)\(\))"
                 r"|(?P<check>sc\.done == 1)"
                 r"|(?P<read>\barrive\(&bars\.(?P<r_id>o_read)\))")


def programs(unit):
    """Role -> its steps within one chunk, from the function `unit`."""
    text = open(SRC).read()
    body = text[text.index(f"void {unit}("):]
    body = body[:body.index("\n}\n")]
    marks = [("chain", "- chain\n"), ("out", "- outputs\n"), ("mma", "- the chain's products\n"),
             ("side", "- products for the output alone\n"), ("", "warp == kKeyWarp")]
    at = [body.index(m) for _, m in marks]
    assert at == sorted(at)
    roles = {}
    for (role, _), a, b in zip(marks, at, at[1:]):
        part = body[a:b]
        part = part[part.index("for (int c = 0; c < nch"):]
        steps = []
        for m in OPS.finditer(part):
            if m["arrive"]:
                steps.append(("arrive", m["a_id"], bool(m["held"])))
            elif m["sync"]:
                steps.append(("sync", m["s_id"], True))
            elif m["wait"]:
                steps.append(("wait", m["w_id"], -1 if "c - 1" in m["phase"] else 0))
            elif m["commit"]:
                steps.append(("commit", m["c_id"], None))
            elif m["past"]:
                # the issuing warp waits from the second chunk on, and once more behind its loop
                steps.append(("arrive", "kBarPast", False) if m["p_kind"] == "arrive" else
                             ("sync", "kBarPast", "not first" if m["later"] else "last"))
            elif m["check"]:
                steps.append(("check", None, None))
            else:
                steps.append(("read", "o_read", None))
        roles[role] = steps
    return roles


class Warp:
    def __init__(self, role, steps, nch):
        self.role, self.steps, self.nch = role, steps, nch
        self.c = self.i = 0
        self.ok, self.inside, self.done = True, None, False

    def step(self):
        return self.steps[self.i]

    def advance(self):
        self.i += 1
        if self.i == len(self.steps):
            self.i, self.c = 0, self.c + 1
            self.done = self.c == self.nch


class Hang(AssertionError):
    pass


def run(roles, nch, rng, bad_record=None, lost=None, last_record=None):
    """bad_record: the chunk whose record says that it is not complete; lost:
    (warp, step, chunk), a wait that runs out although its phase completes;
    last_record: records behind this one never land."""
    warps = [Warp("chain", roles["chain"], nch) for _ in range(CHAIN)]
    warps += [Warp(r, roles[r], nch) for r in ("out", "mma", "side")]
    here = {}  # barrier -> warps that arrived in this phase
    made = {}  # mbarrier -> phases completed

    def landed(name, phase):
        if name in ("key", "tail"):
            return True
        if name == "rec":
            return last_record is None or phase <= last_record
        return phase < 0 or made.get(name, 0) > phase

    def arrive(name, w):
        if w in here.setdefault(name, []):
            raise Hang(f"{w.role} arrives twice in one phase of {name}")
        here[name].append(w)
        if len(here[name]) == (2 if name == "kBarPast" else CHAIN + 1):
            for x in here.pop(name):
                if x.inside == name:
                    x.inside = None
                    x.advance()

    while not all(w.done for w in warps):
        free = []
        for w in warps:
            if w.done or w.inside:
                continue
            kind, name, delta = w.step()
            if kind == "wait" and w.ok and not landed(name, w.c + delta):
                continue
            free.append(w)
        if not free:  # every wait that is bounded runs out
            late = [w for w in warps if not w.done and not w.inside]
            if not late:
                raise Hang(f"nch {nch}: " + ", ".join(f"{w.role}@{w.c} in {w.inside}" for w in warps if not w.done))
            w = rng.choice(late)
            w.ok = False
            if w.role == "out":
                w.done = True
            continue
        w = rng.choice(free)
        kind, name, extra = w.step()
        if (extra == "not first" and w.c == 0) or (extra == "last" and w.c < nch - 1):
            w.advance()
            continue
        if kind == "sync" or (kind == "arrive" and extra and not w.ok):
            w.inside = name
            arrive(name, w)
            continue
        if kind == "arrive":
            arrive(name, w)
        elif kind == "wait":
            if lost and (warps.index(w), w.i, w.c) == lost:
                w.ok = False
                if w.role == "out":  # the output warps leave
                    w.done = True
                    continue
        elif kind == "check":
            if w.c == bad_record:
                w.ok = False
        elif kind in ("commit", "read"):
            if w.ok:
                made[name] = made.get(name, 0) + 1
        w.advance()
    return warps


@pytest.mark.parametrize("unit", ["narrow_unit", "wide_unit"])
def test_every_warp_meets_the_others_whatever_runs_out(unit):
    roles = programs(unit)
    ids = lambda r: [n for k, n, _ in roles[r] if k in ("arrive", "sync") and n != "kBarPast"]  # noqa: E731
    assert sorted(ids("chain")) == sorted(ids("mma") + ids("side")) and len(ids("chain")) == 5
    assert {n for k, n, _ in roles["chain"] if k == "wait"} == {"rec", "x_full", "d_full", "u_full"}
    for seed in range(200):
        rng = random.Random(seed)
        for nch in (1, 2, 5):
            assert all(w.ok for w in run(roles, nch, rng))
            run(roles, nch, rng, bad_record=rng.randrange(nch))
            run(roles, nch, rng, last_record=rng.randrange(-1, nch))
            who = rng.randrange(CHAIN + 3)
            role = ["chain"] * CHAIN + ["out", "mma", "side"]
            waits = [i for i, s in enumerate(roles[role[who]]) if s[0] == "wait"]
            run(roles, nch, rng, lost=(who, rng.choice(waits), rng.randrange(nch)))


def test_nothing_is_under_way_where_a_late_cta_leaves():
    """Read from the source: where a wait has run out, TMEM is given back only
    behind a bounded wait for the products and copies of the CTA."""
    text = open(SRC).read()
    body = lambda name: text[text.index(name):][:text[text.index(name):].index("\n}\n")]  # noqa: E731
    end = body("void end_unit(")
    late = end[end.index("if (bars.timed_out) {"):end.index("tmem_dealloc")]
    assert late.index("mma_commit(bar)") < late.index("warp_wait(bar, 0)") < late.rindex("__syncthreads()")
    chunk = body("gdn_chunk_kernel(const GdnPrefillArgs")
    late = chunk[chunk.index("if (bad && quad == 0) {"):]
    assert max(late.index("warp_wait(&bars[0], 0)"), late.index("warp_wait(&bars[1], 0)")) < late.index("tmem_dealloc")
    early = chunk[:chunk.index("if (bad && quad == 0) {")]
    assert re.search(r"if \(quad == 0 && !bad\) \{\s+tc::tc_fence_after\(\);\s+tc::tmem_dealloc", early)
