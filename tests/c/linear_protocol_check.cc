// The waits of the linear attention kernel (csrc/linear.cu) on the host: every order in
// which its roles, loads and matrix instructions may go on is tried, with the buffers and
// phases of csrc/linear_protocol.h.  Fails where no role can go on before all are done,
// and where something is read that is not what its reader waited for.
//
// A role is a list of steps.  A step waits (for a phase of a barrier, or for a step of another
// role: a load lands after it was issued, a product ends after it was issued), then
// reads and writes buffers and arrives at barriers, all at once.  The warps of a role
// count as one: its barriers count each of them, so a phase waits for the last.
#include <array>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <string>
#include <unordered_set>
#include <vector>

#include "linear_protocol.h"

namespace {

struct Tag {
  int buffer, value;
};
struct Step {
  int bar = -1;                 // phase waited for
  uint32_t parity = 0;
  int role = -1, behind = 0;    // or: `role` is through with this many steps
  std::vector<Tag> reads, writes;
  std::vector<int> arrives;
};
using Role = std::vector<Step>;

struct Model {
  std::vector<Role> roles;
  std::vector<int> need;          // arrivals of a phase, for each barrier
  int buffers = 0;
  int bar(int arrivals) {
    need.push_back(arrivals);
    return (int)need.size() - 1;
  }
  int buffer() { return buffers++; }
  int role() {
    roles.emplace_back();
    return (int)roles.size() - 1;
  }
  Step& add(int r) {
    roles[r].emplace_back();
    return roles[r].back();
  }
  int at(int r) const { return (int)roles[r].size(); }
};

constexpr int kMax = 40;
struct State {
  std::array<uint8_t, kMax> x{};   // steps done of each role, then what each buffer holds
  bool operator==(const State& o) const { return x == o.x; }
};
struct Hash {
  size_t operator()(const State& s) const {
    uint64_t w[kMax / 8], h = 0x9E3779B97F4A7C15ull;
    std::memcpy(w, s.x.data(), kMax);
    for (uint64_t v : w) h = (h ^ v) * 0xD6E8FEB86659FD93ull, h ^= h >> 32;
    return (size_t)h;
  }
};

enum Found { kFine, kStuck, kWrongRead };
const char* name(Found f) { return f == kFine ? "fine" : f == kStuck ? "stuck" : "wrong read"; }

Found explore(const Model& m, size_t* states) {
  const int R = (int)m.roles.size(), B = (int)m.need.size();
  // arrived[r][k][b]: arrivals of role r's first k steps at barrier b.
  std::vector<std::vector<std::vector<int>>> arrived(R);
  for (int r = 0; r < R; ++r) {
    arrived[r].assign(m.roles[r].size() + 1, std::vector<int>(B, 0));
    for (size_t k = 0; k < m.roles[r].size(); ++k) {
      arrived[r][k + 1] = arrived[r][k];
      for (int b : m.roles[r][k].arrives) ++arrived[r][k + 1][b];
    }
  }
  std::unordered_set<State, Hash> seen;
  std::vector<State> todo;
  State first;
  for (int b = 0; b < m.buffers; ++b) first.x[R + b] = 255;
  seen.insert(first);
  todo.push_back(first);
  Found found = kFine;
  while (!todo.empty() && found == kFine) {
    const State s = todo.back();
    todo.pop_back();
    bool moved = false, all = true;
    for (int r = 0; r < R && found == kFine; ++r) {
      if (s.x[r] == m.roles[r].size()) continue;
      all = false;
      const Step& st = m.roles[r][s.x[r]];
      if (st.role >= 0 && s.x[st.role] < st.behind) continue;
      if (st.bar >= 0) {
        int n = 0;
        for (int o = 0; o < R; ++o) n += arrived[o][s.x[o]][st.bar];
        // (the phase of this parity is complete where the current one has the other parity)
        if (((uint32_t)(n / m.need[st.bar]) & 1u) == st.parity) continue;
      }
      moved = true;
      State t = s;
      ++t.x[r];
      for (const Tag& g : st.reads)
        if (s.x[R + g.buffer] != (uint8_t)g.value) found = kWrongRead;
      for (const Tag& g : st.writes) t.x[R + g.buffer] = (uint8_t)g.value;
      if (seen.insert(t).second) todo.push_back(t);
    }
    if (!moved && !all && found == kFine) found = kStuck;
  }
  *states = seen.size();
  return found;
}

// The launch of the segments' end states.  `by_dh`: stages given back by the barriers of dH
// instead of their own, which chunk c + 2 completes again without the producer.  `slots`
// of the scales.
Model state_launch(int chunks, bool by_dh, int slots = dsa::ChunkPipe<true>::scale_slots) {
  using P = dsa::ChunkPipe<true>;
  Model m;
  int full[P::stages], empty[P::stages], v_ready[P::v_bufs], v_free[P::v_bufs], dh_ready[P::dh_bufs], dh_free[P::dh_bufs];
  int kv[P::stages], vt[P::v_bufs], dh[P::dh_bufs];
  for (int i = 0; i < P::stages; ++i) full[i] = m.bar(1), empty[i] = m.bar(P::kv_releases), kv[i] = m.buffer();
  for (int i = 0; i < P::v_bufs; ++i) v_ready[i] = m.bar(1), v_free[i] = m.bar(1), vt[i] = m.buffer();
  for (int i = 0; i < P::dh_bufs; ++i) dh_ready[i] = m.bar(1), dh_free[i] = m.bar(1), dh[i] = m.buffer();
  std::vector<int> scale(slots);
  for (int& i : scale) i = m.buffer();
  const int producer = m.role(), issuer = m.role(), tensor = m.role(), state = m.role();
  int land[P::stages], decay[3];
  for (int& r : land) r = m.role();
  for (int& r : decay) r = m.role();
  for (int c = 0; c < chunks; ++c) {
    const int s = P::stage(c), d = P::dh(c);
    const int scaled = scale[slots == P::scale_slots ? P::scale(c) : c % slots];
    Step& load = m.add(producer);
    if (c >= P::stages) {
      const int last = c - P::stages;
      load.bar = by_dh ? dh_ready[P::dh(last)] : empty[s];
      load.parity = by_dh ? P::dh_phase(last) : P::stage_phase(last);
    }
    load.writes = {{kv[s], c}};
    Step& lands = m.add(land[s]);
    lands.role = producer, lands.behind = m.at(producer);
    lands.arrives = {full[s]};
    if (c >= P::dh_bufs) {
      Step& w = m.add(issuer);
      w.bar = dh_free[d], w.parity = P::dh_phase(c - P::dh_bufs);
    }
    for (int g = 0; g < 4; ++g) {
      const int b = P::v(g), who = decay[(4 * c + g) % 3];
      Step& seen = m.add(who);
      seen.bar = full[s], seen.parity = P::stage_phase(c);
      Step& w = m.add(who);
      if (!P::v_first(c, g)) w.bar = v_free[b], w.parity = P::v_phase_before(c, g);
      w.reads = {{kv[s], c}};
      w.writes = {{vt[b], 4 * c + g}};
      if (g == 0) w.writes.push_back({scaled, c});
      w.arrives = {v_ready[b]};
      Step& issue = m.add(issuer);
      issue.bar = v_ready[b], issue.parity = P::v_phase(c, g);
      Step& ends = m.add(tensor);
      ends.role = issuer, ends.behind = m.at(issuer);
      ends.reads = {{kv[s], c}, {vt[b], 4 * c + g}};
      ends.writes = {{dh[d], g < 3 ? 254 : c}};
      ends.arrives = {v_free[b]};
      if (g == 3) ends.arrives.insert(ends.arrives.end(), {dh_ready[d], empty[s]});
    }
    Step& r = m.add(state);
    r.bar = dh_ready[d], r.parity = P::dh_phase(c);
    Step& takes = m.add(state);
    takes.reads = {{dh[d], c}, {scaled, c}};
    takes.arrives = {dh_free[d]};
  }
  return m;
}

// The launch of the outputs.  `tiles` barriers for the staged output tiles, in turn.
Model output_launch(int chunks, int tiles) {
  using P = dsa::ChunkPipe<false>;
  constexpr int kStaged = 100;   // an output tile over chunk c's Q holds kStaged + c
  Model m;
  int kv_full[P::stages], kv_empty[P::stages], q_full[P::stages], q_empty[P::stages], kv[P::stages], q[P::stages];
  int v_ready[P::v_bufs], v_free[P::v_bufs], vt[P::v_bufs], scale[P::scale_slots];
  for (int i = 0; i < P::stages; ++i) {
    kv_full[i] = m.bar(1), kv_empty[i] = m.bar(P::kv_releases), q_full[i] = m.bar(1), q_empty[i] = m.bar(1);
    kv[i] = m.buffer(), q[i] = m.buffer();
  }
  for (int i = 0; i < P::v_bufs; ++i) v_ready[i] = m.bar(1), v_free[i] = m.bar(1), vt[i] = m.buffer();
  for (int& i : scale) i = m.buffer();
  std::vector<int> staged(tiles);
  for (int& i : staged) i = m.bar(1);
  const int s_ready = m.bar(1), qh_ready = m.bar(1), h_ready = m.bar(1), p_ready = m.bar(1), o_ready = m.bar(1);
  const int o_free = m.bar(1), dh_ready = m.bar(1), dh_free = m.bar(1);
  const int sp = m.buffer(), o = m.buffer(), hb = m.buffer(), dh = m.buffer();   // S and P, O, H, dH
  const int producer = m.role(), out = m.role(), out_tensor = m.role(), delta = m.role(), delta_tensor = m.role();
  const int rows = m.role(), decay = m.role(), state = m.role(), store = m.role();
  int kv_land[P::stages], q_land[P::stages];
  for (int i = 0; i < P::stages; ++i) kv_land[i] = m.role(), q_land[i] = m.role();
  auto wait = [&](int r, int bar, uint32_t parity) -> Step& {
    Step& s = m.add(r);
    s.bar = bar, s.parity = parity;
    return s;
  };
  auto follows = [&](int r, int other) -> Step& {   // behind what `other` has done so far
    Step& s = m.add(r);
    s.role = other, s.behind = m.at(other);
    return s;
  };
  for (int c = 0; c < chunks; ++c) {
    const int s = P::stage(c), last = c - P::stages;
    const uint32_t odd = (uint32_t)c & 1u;
    Step& k_load = m.add(producer);
    if (c >= P::stages) k_load.bar = kv_empty[s], k_load.parity = P::stage_phase(last);
    k_load.writes = {{kv[s], c}};
    follows(kv_land[s], producer).arrives = {kv_full[s]};
    Step& q_load = m.add(producer);
    if (c >= P::stages) q_load.bar = q_empty[s], q_load.parity = P::stage_phase(last);
    q_load.writes = {{q[s], c}};
    follows(q_land[s], producer).arrives = {q_full[s]};

    wait(out, kv_full[s], P::stage_phase(c));
    wait(out, q_full[s], P::stage_phase(c));
    Step& ends_s = follows(out_tensor, out);
    ends_s.reads = {{kv[s], c}, {q[s], c}}, ends_s.writes = {{sp, c}}, ends_s.arrives = {s_ready};
    wait(out, h_ready, odd);
    if (c > 0) wait(out, o_free, odd ^ 1u);
    Step& ends_h = follows(out_tensor, out);
    ends_h.reads = {{q[s], c}, {hb, c}}, ends_h.writes = {{o, c}}, ends_h.arrives = {qh_ready};
    wait(out, p_ready, odd);
    Step& ends_p = follows(out_tensor, out);
    ends_p.reads = {{kv[s], c}, {sp, kStaged + c}, {o, kStaged + c}};
    ends_p.writes = {{o, c}}, ends_p.arrives = {o_ready, kv_empty[s]};

    wait(rows, s_ready, odd).reads = {{sp, c}};
    Step& p = wait(rows, qh_ready, odd);
    p.reads = {{o, c}}, p.writes = {{sp, kStaged + c}, {o, kStaged + c}}, p.arrives = {p_ready};
    Step& tile = wait(rows, o_ready, odd);
    tile.reads = {{o, c}}, tile.writes = {{q[s], kStaged + c}};
    tile.arrives = {o_free, staged[c % tiles]};
    wait(store, staged[c % tiles], (uint32_t)(c / tiles) & 1u);
    Step& stored = m.add(store);
    stored.reads = {{q[s], kStaged + c}}, stored.arrives = {q_empty[s]};

    if (c > 0) wait(delta, dh_free, P::dh_phase(c - 1));
    for (int g = 0; g < 4; ++g) {
      const int b = P::v(g);
      if (g == 0) wait(decay, kv_full[s], P::stage_phase(c));
      Step& w = m.add(decay);
      if (!P::v_first(c, g)) w.bar = v_free[b], w.parity = P::v_phase_before(c, g);
      w.reads = {{kv[s], c}}, w.writes = {{vt[b], 4 * c + g}}, w.arrives = {v_ready[b]};
      if (g == 0) w.writes.push_back({scale[P::scale(c)], c});
      wait(delta, v_ready[b], P::v_phase(c, g));
      Step& ends = follows(delta_tensor, delta);
      ends.reads = {{kv[s], c}, {vt[b], 4 * c + g}}, ends.writes = {{dh, g < 3 ? 254 : c}}, ends.arrives = {v_free[b]};
      if (g == 3) ends.arrives.insert(ends.arrives.end(), {dh_ready, kv_empty[s]});
    }
    Step& h = m.add(state);
    if (c > 0) h.bar = qh_ready, h.parity = odd ^ 1u;
    h.writes = {{hb, c}}, h.arrives = {h_ready};
    wait(state, dh_ready, P::dh_phase(c));
    Step& takes = m.add(state);
    takes.reads = {{dh, c}, {scale[P::scale(c)], c}}, takes.arrives = {dh_free};
  }
  return m;
}

int failed = 0;
void expect(const char* what, const Model& m, Found want) {
  if (m.roles.size() + m.buffers > kMax) {
    std::printf("FAIL %s: too many roles and buffers\n", what);
    ++failed;
    return;
  }
  size_t n = 0;
  const Found f = explore(m, &n);
  std::printf("%s %s: %s (%zu states)\n", f == want ? "ok" : "FAIL", what, name(f), n);
  failed += f != want;
}

}  // namespace

int main() {
  expect("states' launch", state_launch(7, false), kFine);
  expect("states' launch, stages given back by the barriers of dH", state_launch(7, true), kStuck);
  expect("states' launch, two slots of scales", state_launch(7, false, 2), kWrongRead);
  expect("outputs' launch", output_launch(5, dsa::ChunkPipe<false>::o_tiles), kFine);
  expect("outputs' launch, one barrier for the staged output tiles", output_launch(5, 1), kStuck);
  if (!failed) std::printf("all ok\n");
  return failed != 0;
}
