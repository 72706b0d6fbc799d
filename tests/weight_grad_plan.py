"""Which tiles and how many splits zf_weight_grad takes for given sizes: its plan, with the numbers read from the source,
so that tests of a form can say that their cases still reach it."""
import os
import re

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fsdp_sharded_mixed_amd", "csrc",
                      "zf_weight_grad.hip")
FORMS = ("big", "middle", "little")


def _numbers(pattern, text):
    found = re.search(pattern, text)
    assert found, f"the plan is written in another way now: {pattern}"
    return [float(v) for v in found.groups()]


def read():
    with open(SOURCE) as f:
        text = re.sub(r"\s+", " ", f.read())
    n, forms = r"([\d.]+)", {}
    for form, v in zip(FORMS, "bml"):
        bm, bn = _numbers(rf"typedef Tile<{n}, {n}, \d, \d> {form.capitalize()};", text)
        if form == "big":
            places, least = _numbers(rf"s{v} = splits_of\(rows, {form}, {n}, {n}\)", text)
            ragged = least  # not taken without whole pieces
        else:
            places, least, ragged = _numbers(rf"s{v} = splits_of\(rows, {form}, {n}, whole \? {n} : {n}\)", text)
        room, stage, more = _numbers(rf"c{v} = cost\(rows, out \* in, {form}, s{v}, {n}, {n}, {n}\)", text)
        forms[form] = dict(bm=int(bm), bn=int(bn), places=int(places), least=int(least), ragged=int(ragged),
                           room=int(room), stage=stage, more=more)
    depth = _numbers(rf"kStages = \d+, kDepth = {n};", text)[0]
    join, rate = _numbers(rf"splits > 1 \? {n} \+ \(double\)\(splits \* size\) \* 4 / ([\de.]+) : 0", text)
    return forms, int(depth), join, rate


def chosen(rows, outs, ins, whole=True):
    """(form, splits)."""
    forms, depth, join, rate = read()
    best = None
    for form in ("little", "middle", "big"):  # an equal cost keeps the later of the first two, and them before the last
        f = forms[form]
        if form == "big" and not whole:
            continue
        tiles = -(-outs // f["bm"]) * -(-ins // f["bn"])
        splits = max(1, min(f["places"] // tiles, rows // (f["least"] if whole else f["ragged"])))
        rounds = -(-tiles * splits // f["room"])
        us = rounds * (-(-rows // (splits * depth)) * f["stage"] + f["more"]) \
            + (join + splits * outs * ins * 4 / rate if splits > 1 else 0)
        if best is None or us < best[0] or (us == best[0] and form == "middle"):
            best = (us, form, splits)
    stages = -(-rows // depth)
    per = max(1, -(-stages // best[2]))
    return best[1], max(1, -(-stages // per))


# Whole numbers whose exact sums the tests of the largest tiles compare with: one split, so that the tiles are stored
# into or added to the gradient itself; rows, out, in, all of which end inside a stage or a tile.
LARGE = [(2117, 2824, 2832), (289, 2824, 2832), (1003, 2312, 3600)]
