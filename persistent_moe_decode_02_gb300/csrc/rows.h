// How the rows of probabilities and verifications (verify.cu) are split over
// blocks.  Plain host code.
#pragma once

namespace mk {

constexpr int ROW_THREADS = 512;
constexpr int MANY = 8, FEW = 16;             // blocks of a row's cluster at most: of many rows, of few
constexpr int STEP = ROW_THREADS * 4;         // elements of one pass of a block: 4 consecutive ones a thread
constexpr int MAX_PASSES = 24;                // kept in registers: 96 of a thread
constexpr int MAX_VOCAB = MANY * MAX_PASSES * STEP;   // 393216

// Blocks of a row's cluster on a device of `sms` multiprocessors, `most` at
// most.  Few rows, whose blocks all have an SM of their own, are split as far
// as a pass for each block, into 16 at most (beyond what every device has to
// offer, so asked for; where it is not, `most` is 8): of 151936, 1 row takes
// 4.2 us of probabilities and 5.5 of verification then instead of 4.9 and 7.4
// with 8, 9 rows 5.6 and 7.1 instead of 5.2 and 7.7.  Of many rows a block
// takes four passes before the row is split further, into 8 at most (160 rows
// of 32000: 9.8 us, 14.4 when split down to a pass; 120 of 9000: 3.8 and 11.1;
// 16 verifications of 151936: 9.2 us, 12.2 with 16 blocks a row when one of 8
// took 10.9).
inline int cluster_of(int vocab, long long rows, int sms, int most) {
  const bool few = rows * FEW <= sms;
  if (!few && most > MANY) most = MANY;
  int c = 1;
  while (c < most && vocab > c * STEP * (few ? 1 : 4)) c *= 2;
  return c;
}

// Elements of a block's segment at most, and passes over it.
inline int segment_of(int vocab, int cluster) { return ((vocab + cluster - 1) / cluster + 3) / 4 * 4; }
inline int passes_of(int vocab, int cluster) { return (segment_of(vocab, cluster) + STEP - 1) / STEP; }

// Blocks that run at once when two share an SM, as a multiple of every
// cluster's size: a block fetches ahead for the one that many later.
inline int blocks_at_once(int sms) { return 2 * sms / FEW * FEW; }

}  // namespace mk
