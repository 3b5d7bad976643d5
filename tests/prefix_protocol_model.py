"""Executable model of the synchronisation protocol of the long-prefix kernel
(dynamic_hierarchical_sparse_b200/csrc/paged_prefix.cu).

A CTA works on pieces, each of some key tiles. Its roles are restated as
sequential programs, in the kernel's order:

* the K and the V producer: tile n (counted across pieces) into slot n % stages,
  once the tile before in that slot is released;
* an MMA-issuing thread for each lane. Two lanes (d 64, 128) take turns; a turn
  is P V of the lane's last tile, then S of its next one over the same TMEM
  columns. One lane (d 256) has two places for S and P and issues S of the next
  tile first. Lanes on the same rows (`apart`) take every other tile, and a
  tile's owner releases it for both;
* four softmax warps a lane: send for Q, read S, write P in two halves, rescale O
  in between, hand P over, and at a piece's end read O (apart: both lanes' O, with
  (m, l) crossing in TMEM) before the next piece's products start.

The driver and the phase checks are those of pair_protocol_model.Model.

Checked: no deadlock; phase integrity; K, V and Q read only once there; S and P
places overwritten only when read; P complete before its products; O rescaled only
between two tiles' products, read only after a piece's last, overwritten only when
read; Q rewritten only after the last S that reads it.
"""

from __future__ import annotations

import dataclasses
import random
from typing import List, Optional

from pair_protocol_model import Model, ProtocolViolation, _Barrier


@dataclasses.dataclass(frozen=True)
class Piece:
    count: int         # key tiles
    apart: bool        # lanes take every other tile (two lanes only)
    valid: tuple       # per lane: the warps that have a valid row
    edge: bool         # its last tile ends inside


@dataclasses.dataclass(frozen=True)
class PrefixMutation:
    """Protocol slips (each off by default)."""
    one_place_barriers: bool = False   # one lane: one barrier for both places of S and P
    rescale_without_wait: bool = False # one lane: O rescaled without waiting for the last tile's products
    s_first: bool = False              # two lanes: S of the next tile before P V
    no_piece_barrier: bool = False     # two lanes: the next piece starts when a lane's own warp is done
    release_once: bool = False         # apart: the owner's release does not stand for the other lane
    q_early: bool = False              # the next piece's Q sent for before the last S is done
    no_cross_wait: bool = False        # apart: the other lane's results read without waiting
    half_for_full: bool = False        # the second half of P V issued on the first half's arrival


class PrefixModel(Model):
    def __init__(self, pieces: List[Piece], lanes: int, k_stages: int, v_stages: int,
                 mut: PrefixMutation = PrefixMutation(), rescale_prob: float = 0.5,
                 rng: Optional[random.Random] = None):
        self.pieces, self.lanes, self.ks, self.vs, self.pmut = pieces, lanes, k_stages, v_stages, mut
        self.rescale_prob = rescale_prob
        self.rng = rng or random.Random(0)
        B = self.bars = {}
        for s in range(k_stages):
            B["KFull%d" % s], B["KFree%d" % s] = _Barrier("KFull%d" % s, 1), _Barrier("KFree%d" % s, lanes)
        for s in range(v_stages):
            B["VFull%d" % s], B["VFree%d" % s] = _Barrier("VFull%d" % s, 1), _Barrier("VFree%d" % s, lanes)
        for x in (0, 1):
            for name, count in (("SFull", 1), ("PHalf", 4), ("PFull", 4), ("QFull", 4), ("ODone", 1), ("Turn", 1),
                                ("Cross", 4)):
                B[name + str(x)] = _Barrier(name + str(x), count)
        B["Piece"] = _Barrier("Piece", 4 * lanes)
        self.smem = {"K%d" % s: [None, 0] for s in range(k_stages)}
        self.smem.update({"V%d" % s: [None, 0] for s in range(v_stages)})
        self.tma, self.queues, self.waiting = [], {0: [], 1: []}, {}
        self.Q = {a: [None] * 4 for a in range(lanes)}            # piece of each warp's rows
        self.s_left = {}                                          # (lane, piece): S products not yet done
        for a in range(lanes):
            for i, p in enumerate(pieces):
                self.s_left[a, i] = len(self._tiles(p, a))
        self.place = {x: None for x in (0, 1)}                    # S and P
        self.cross = {x: set() for x in (0, 1)}                   # readers that (m, l) in a place still waits for
        self.O = {a: {"piece": None, "done": [], "unread": set()} for a in range(lanes)}
        self.roles = {"prodK": self._prod("K", k_stages), "prodV": self._prod("V", v_stages)}
        for a in range(lanes):
            self.roles["mma%d" % a] = self._mma(a)
            for w in range(4):
                self.roles["smx%d.%d" % (a, w)] = self._softmax(a, w)
        self.pending_op = {r: None for r in self.roles}
        self.finished = set()

    # --------------------------------------------------------------- helpers
    def _tiles(self, p: Piece, a: int):
        return list(range(a, p.count, 2)) if p.apart else list(range(p.count))

    def _at(self, a: int, m: int):
        """(place and barrier, phase) of a lane's tile m."""
        if self.lanes == 2:
            return a, m
        return m & 1, m >> 1

    def _bar(self, a: int, m: int):
        if self.lanes == 1 and self.pmut.one_place_barriers:
            return 0, m
        return self._at(a, m)

    # --------------------------------------------------------------- roles
    def _prod(self, kind: str, stages: int):
        for n in range(sum(p.count for p in self.pieces)):
            s, r = n % stages, n // stages
            if r > 0:
                yield ("wait", "%sFree%d" % (kind, s), r - 1)
            yield ("expect", "%sFull%d" % (kind, s), r, "prod", 1)
            yield ("tma", "%s%d" % (kind, s), n, "%sFull%d" % (kind, s))

    def _mma(self, a: int):
        n0 = mine = sent = turn = ends = 0
        for i, p in enumerate(self.pieces):
            tiles = self._tiles(p, a)
            turns = 1 + ((p.count + 1) // 2 if p.apart else p.count)
            yield ("wait", "QFull%d" % a, i)
            for x in range(turns):
                pv = tiles[x - 1] if 0 < x <= len(tiles) else None
                sn = tiles[x] if x < len(tiles) else None
                last = pv is not None and sn is None

                def k_there():
                    yield ("wait", "KFull%d" % ((n0 + sn) % self.ks), (n0 + sn) // self.ks)

                def p_there():
                    b, ph = self._bar(a, mine)
                    yield ("wait", "VFull%d" % ((n0 + pv) % self.vs), (n0 + pv) // self.vs)
                    yield ("wait", "PHalf%d" % b, ph)

                def send_s():
                    b, ph = self._bar(a, sent)
                    yield ("mma", a, "S", self._at(a, sent)[0], i, n0 + sn)
                    yield ("commit", a, "SFull%d" % b, ph, "")

                def send_pv():
                    b, ph = self._bar(a, mine)
                    yield ("mma", a, "PV", self._at(a, mine)[0], i, n0 + pv, 0, x == 1)
                    if not self.pmut.half_for_full:
                        yield ("wait", "PFull%d" % b, ph)
                    yield ("mma", a, "PV", self._at(a, mine)[0], i, n0 + pv, 1, False)
                    if self.pmut.half_for_full:
                        yield ("wait", "PFull%d" % b, ph)

                def release(kind, stages, n):
                    twice = p.apart and not self.pmut.release_once
                    for who in ["", "+"] if twice else [""]:
                        yield ("commit", a, "%sFree%d" % (kind, n % stages), n // stages, who)

                if self.lanes == 2:
                    if pv is not None:
                        yield from p_there()
                    if sn is not None:
                        yield from k_there()
                    if a == 1:
                        yield ("wait", "Turn0", turn)
                    elif turn > 0:
                        yield ("wait", "Turn1", turn - 1)
                    if self.pmut.s_first and sn is not None:
                        yield from send_s()
                    if pv is not None:
                        yield from send_pv()
                    if sn is not None and not self.pmut.s_first:
                        yield from send_s()
                    yield ("arrive", "Turn%d" % a, turn, "mma%d" % a)
                    if sn is not None:
                        yield from release("K", self.ks, n0 + sn)
                else:
                    if sn is not None:
                        yield from k_there()
                        yield from send_s()
                        yield from release("K", self.ks, n0 + sn)
                    if pv is not None:
                        yield from p_there()
                        yield from send_pv()
                if sn is not None:
                    sent += 1
                if pv is not None:
                    if last:
                        yield ("commit", a, "ODone%d" % a, ends, "")
                        ends += 1
                    yield from release("V", self.vs, n0 + pv)
                    mine += 1
                turn += 1
            n0 += p.count

    def _softmax(self, a: int, w: int):
        me = "smx%d.%d" % (a, w)
        n0 = mine = ends = joins = 0
        yield ("q_write", a, w, 0)
        for i, p in enumerate(self.pieces):
            more = i + 1 < len(self.pieces)
            valid = w in p.valid[a]
            yield ("arrive", "QFull%d" % a, i, me)
            tiles = self._tiles(p, a)
            if self.pmut.q_early and more and tiles:
                yield ("q_write", a, w, i + 1)
            for x, kt in enumerate(tiles):
                at, _ = self._at(a, mine)
                b, ph = self._bar(a, mine)
                n = n0 + kt
                yield ("wait", "SFull%d" % b, ph)
                if p.edge and kt == p.count - 1:
                    yield ("wait", "VFull%d" % (n % self.vs), n // self.vs)
                if valid:
                    yield ("read_S", at, a, w, n)
                    yield ("write_P", at, a, w, n, 0)
                    if x > 0 and self.rng.random() < self.rescale_prob:
                        if self.lanes == 1 and not self.pmut.rescale_without_wait:
                            yield ("wait", "VFree%d" % ((n - 1) % self.vs), (n - 1) // self.vs)
                        yield ("rescale", a, i, tiles[:x])
                yield ("arrive", "PHalf%d" % b, ph, me)
                if valid:
                    yield ("write_P", at, a, w, n, 1)
                yield ("arrive", "PFull%d" % b, ph, me)
                mine += 1
            if more and not (self.pmut.q_early and tiles):
                yield ("q_write", a, w, i + 1)
            if tiles:
                yield ("wait", "ODone%d" % a, ends)
                ends += 1
            if not p.apart:
                if valid:
                    yield ("read_O", a, a, w, i)
            else:
                yield ("cross_write", a, w, i)
                yield ("arrive", "Cross%d" % a, joins, me)
                if not self.pmut.no_cross_wait:
                    yield ("wait", "Cross%d" % (1 - a), joins)
                if valid:
                    yield ("cross_read", a, w)
                    yield ("read_O", 0, a, w, i)
                    if p.count > 1:
                        yield ("read_O", 1, a, w, i)
                joins += 1
            if self.lanes == 2 and more and not self.pmut.no_piece_barrier:
                yield ("arrive", "Piece", i, me)
                yield ("wait", "Piece", i)
            n0 += p.count

    # -------------------------------------------------------------- ops
    def _run_sync(self, role, op):
        kind = op[0]
        if kind == "q_write":
            _, a, w, i = op
            if i > 0 and self.s_left[a, i - 1]:
                raise ProtocolViolation("Q of lane %d rewritten for piece %d with %d S products to come"
                                        % (a, i, self.s_left[a, i - 1]))
            self.Q[a][w] = i
            return True
        if kind == "read_S":
            _, at, a, w, n = op
            S = self.place[at]
            if S is None or S["tag"] != (a, n):
                raise ProtocolViolation("%s reads S of tile %d, finds %s" % (role, n, S and S["tag"]))
            S["readers"].add(w)
            return True
        if kind == "write_P":
            _, at, a, w, n, half = op
            S = self.place[at]
            if S["tag"] != (a, n) or w not in S["readers"]:
                raise ProtocolViolation("%s writes P of tile %d over %s" % (role, n, S["tag"]))
            S["P"].add((w, half))
            return True
        if kind == "rescale":
            _, a, i, tiles = op
            if self.O[a]["piece"] != i or len(self.O[a]["done"]) != 2 * len(tiles):
                raise ProtocolViolation("%s rescales O of piece %d behind %d tiles: %s" % (role, i, len(tiles), self.O[a]))
            return True
        if kind == "read_O":
            _, b, a, w, i = op
            p = self.pieces[i]
            if self.O[b]["piece"] != i or len(self.O[b]["done"]) != 2 * len(self._tiles(p, b)):
                raise ProtocolViolation("%s reads O %d of piece %d: %s" % (role, b, i, self.O[b]))
            self.O[b]["unread"].discard((a, w))
            return True
        if kind == "cross_write":
            _, a, w, i = op
            p = self.pieces[i]
            S = self.place[a]
            if S is not None and len(S["pv"]) != 2:
                raise ProtocolViolation("%s writes (m, l) over P of %s" % (role, S["tag"]))
            self.crossed = getattr(self, "crossed", set())
            self.crossed.add((a, w, i))
            if w in p.valid[1 - a]:
                self.cross[a].add(w)
            return True
        if kind == "cross_read":
            _, a, w = op
            if w not in self.cross[1 - a]:
                raise ProtocolViolation("%s reads (m, l) of the other lane before they are there" % role)
            self.cross[1 - a].discard(w)
            return True
        return super()._run_sync(role, op)

    def _exec_mma(self, a: int) -> None:
        op = self.queues[a].pop(0)
        if op[0] == "commit":
            self.bars[op[2]].arrive("mma%d%s" % (a, op[4]), op[3], self)
            return
        if op[2] == "S":
            _, _, _, at, i, n = op
            if any(q != i for q in self.Q[a]):
                raise ProtocolViolation("S of tile %d reads Q rows of pieces %s" % (n, self.Q[a]))
            self._read_smem("K%d" % (n % self.ks), n)
            S = self.place[at]
            if S is not None:
                if not set(S["valid"]) <= S["readers"]:
                    raise ProtocolViolation("S of tile %d over S of %s, read by %s" % (n, S["tag"], S["readers"]))
                if len(S["pv"]) != 2:
                    raise ProtocolViolation("S of tile %d over P of %s before its products" % (n, S["tag"]))
            if self.cross[at]:
                raise ProtocolViolation("S of tile %d over (m, l) that warps %s have not read" % (n, self.cross[at]))
            self.place[at] = {"tag": (a, n), "readers": set(), "P": set(), "pv": set(),
                              "valid": self.pieces[i].valid[a]}
            self.s_left[a, i] -= 1
            return
        _, _, _, at, i, n, half, new = op
        self._read_smem("V%d" % (n % self.vs), n)
        S = self.place[at]
        if S["tag"] != (a, n) or any((w, half) not in S["P"] for w in S["valid"]):
            raise ProtocolViolation("P V of tile %d, half %d: place holds %s" % (n, half, S))
        S["pv"].add(half)
        O = self.O[a]
        if new:
            if O["unread"]:
                raise ProtocolViolation("P V of piece %d over O of piece %s, not read by %s" % (i, O["piece"], O["unread"]))
            p = self.pieces[i]
            unread = {(b, w) for b in range(self.lanes) for w in p.valid[b]} if p.apart else {(a, w) for w in p.valid[a]}
            self.O[a] = O = {"piece": i, "done": [], "unread": unread}
        O["done"].append((n, half))


def random_pieces(rng: random.Random, lanes: int, most: int = 4, tiles: int = 7) -> List[Piece]:
    """Pieces as the work list forms them: rows of a tile fill its first warps."""
    out = []
    for _ in range(rng.randint(1, most)):
        apart = lanes == 2 and rng.random() < 0.5
        if apart or lanes == 1:
            v = tuple(range(rng.randint(1, 4)))
            valid = (v, v) if lanes == 2 else (v,)
        else:
            valid = (tuple(range(4)), tuple(range(rng.randint(1, 4))))
        out.append(Piece(rng.randint(1, tiles), apart, valid, rng.random() < 0.4))
    return out
